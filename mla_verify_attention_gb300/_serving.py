"""Bindings of the grouped-head verify attention and of the cache operators.

Argument marshalling only, as in ``_lib``: shapes, types and devices are
checked, addresses and strides passed on, and a status other than MLA_OK
raises ``MLAError``.  Problems only the GPU can see are in
``last_device_error``.
"""
from __future__ import annotations

import ctypes
import struct

from ._lib import MLA_OK, MLAError, empty_on, load_library

_STRIDES = ctypes.c_longlong * 9
LATENT, ROPE, ROW = 512, 64, 576

# A verify step makes several of these calls, each a few microseconds of GPU
# time, so they are kept as lean as checks allow: arguments are packed into one
# array (ctypes takes 1.3 us to convert sixteen of them, 0.4 us for this), and
# what is looked up once is bound by the first call.
_EXTEND, _TRIM, _APPEND, _KEEP, _GQA, _GQA_PAGED = range(6)
_WINDOW, _WINDOW_PAGED, _APPEND_FP4, _SELECT, _COMPACT, _WEIGHTS, _WEIGHTS_PAGED, _FP4_PAGED = range(8, 16)
_pack_extend = struct.Struct("=13q").pack
_pack_trim = struct.Struct("=10q").pack
_pack_append = struct.Struct("=14q").pack
_pack_keep = struct.Struct("=16q").pack
_pack_gqa = struct.Struct("=13qd5q").pack
_pack_paged = struct.Struct("=16qd5q").pack
_pack_window = struct.Struct("=13qd7q").pack
_pack_window_paged = struct.Struct("=16qd7q").pack
_pack_append_fp4 = struct.Struct("=7q2d12q").pack
_pack_fp4_paged = struct.Struct("=18q3d5q").pack
_pack_select = struct.Struct("=13q").pack
_pack_compact = struct.Struct("=18q").pack
_pack_weights = struct.Struct("=13qd2q").pack
_pack_weights_paged = struct.Struct("=16qd2q").pack

_torch = _call = None
_current_device = _current_stream = _int32 = _bf16 = _fp16 = _fp32 = _uint8 = None


def _bind():
    global _torch, _call, _current_device, _current_stream, _int32, _bf16, _fp16, _fp32, _uint8
    import torch
    _torch, _int32 = torch, torch.int32
    _bf16, _fp16, _fp32, _uint8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
    if hasattr(torch._C, "_cuda_getDevice"):
        _current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    else:                                        # a torch without CUDA: no tensor gets past the device check
        _current_device = _current_stream = lambda *_: -2
    _call = load_library().mla_call_packed


def _wrong_device(*tensors):
    if not all(t.is_cuda for t in tensors):
        raise ValueError("expected CUDA tensors")
    if len({t.get_device() for t in tensors}) > 1:
        raise ValueError("all tensors must be on one device")
    raise ValueError("the tensors' device must be the current one")


def _on_current(dev):
    return dev >= 0 and dev == _current_device()


def _handle(stream, dev):
    return _current_stream(dev) if stream is None else int(stream.cuda_stream)


def _empty(shape, dt, like, stream, result=True):
    """Memory that a call on `stream` writes, out of that stream's pool."""
    if stream is None:
        return _torch.empty(shape, dtype=dt, device=like.device)
    return empty_on(stream, shape, dt, like.device, result)


def _ints(name, t, *shape):
    if t.dtype is not _int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s" % (name, list(shape)))


def _wrong_ints(**tensors):
    for name, (t, *shape) in tensors.items():
        _ints(name, t, *shape)


# ---------------------------------------------------------------- attention

def gqa_workspace_size(B: int, q_len: int, H: int, Hkv: int, D: int) -> int:
    """Workspace bytes of the two calls below on the current device."""
    return int(load_library().mla_gqa_workspace_size(B, q_len, H, Hkv, D))


def _gqa(q, k, v, seq_lens, tree_mask, out, lse, workspace, Hkv, stream):
    B, q_len, H, D = q.shape
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt or (dt is not _bf16 and dt is not _fp16):
        raise ValueError("q, k and v must have one type, bfloat16 or float16")
    _ints("seq_lens", seq_lens, B)
    if (tree_mask.element_size() != 4 or tree_mask.shape != (B, q_len, (q_len + 31) >> 5)
            or not tree_mask.is_contiguous() or tree_mask.is_floating_point()):
        raise ValueError("tree_mask must be contiguous 32-bit words [B,q,ceil(q/32)]")
    strides = 0
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        if qs[3] != 1 or ks[-1] != 1 or vs[-1] != 1:
            raise ValueError("the innermost dimension of q, k and v must be contiguous")
        if len(ks) == 3:            # pools: no batch dimension
            ks, vs = (8,) + ks, (8,) + vs
        strides = _STRIDES(*qs[:3], *ks[:3], *vs[:3])
    if out is None:
        out = _empty((B, q_len, H, D), dt, q, stream)
    elif out.dtype is not dt or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is None:
        lse = _empty((B, q_len, H), _fp32, q, stream)
    elif lse.dtype is not _fp32 or lse.shape != (B, q_len, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,q,H]")
    if workspace is None:
        workspace = _empty(gqa_workspace_size(B, q_len, H, Hkv, D), _torch.uint8, q, stream, result=False)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return B, q_len, H, D, 0 if dt is _bf16 else 1, strides, out, lse, workspace


def gqa_verify_attn(q, k, v, seq_lens, tree_mask, scale, out=None, lse=None, workspace=None, stream=None):
    """Verify attention with grouped query heads on the current CUDA device.

    q [B,q,H,D], k and v [B,Smax,Hkv,D], bf16 or fp16, D 64 or 128, H a
    multiple of Hkv; strided views are taken as they are if the innermost
    dimension is contiguous.  seq_lens [B] int32 counts the drafts' own rows
    (0: unused stream), tree_mask [B,q,ceil(q/32)] as for ``verify_attn``.
    Returns (out [B,q,H,D] in q's type, lse [B,q,H] fp32); a row whose mask
    leaves nothing has out 0 and lse -inf.  Without out, lse or workspace they
    are made, out of `stream`'s own pool where that is another stream.
    """
    if _call is None:
        _bind()
    shape = k.shape
    if q.dim() != 4 or len(shape) != 4 or v.shape != shape or shape[0] != q.shape[0] or shape[3] != q.shape[3]:
        raise ValueError("expected q [B,q,H,D], k and v [B,Smax,Hkv,D]")
    dev = q.get_device()
    if not (_on_current(dev) and dev == k.get_device() == v.get_device() == seq_lens.get_device()
            == tree_mask.get_device()):
        _wrong_device(q, k, v, seq_lens, tree_mask)
    B, q_len, H, D, dt, strides, out, lse, ws = _gqa(q, k, v, seq_lens, tree_mask, out, lse, workspace, shape[2],
                                                     stream)
    if not dev == out.get_device() == lse.get_device() == ws.get_device():
        _wrong_device(q, out, lse, ws)
    st = _call(_GQA, _pack_gqa(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides and ctypes.addressof(strides), seq_lens.data_ptr(),
        tree_mask.data_ptr(), B, q_len, H, shape[2], D, shape[1], dt, scale, out.data_ptr(), lse.data_ptr(),
        ws.data_ptr(), ws.numel() * ws.element_size(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_verify_attn")
    return out, lse


def gqa_verify_attn_paged(q, k_pool, v_pool, block_table, page_size, seq_lens, tree_mask, scale, out=None, lse=None,
                          workspace=None, stream=None):
    """gqa_verify_attn over pools k_pool, v_pool [pool_rows,Hkv,D] of pages of
    page_size >= 1 rows, block_table [B,max_blocks] int32; read in place."""
    if _call is None:
        _bind()
    shape = k_pool.shape
    if (q.dim() != 4 or len(shape) != 3 or v_pool.shape != shape or shape[2] != q.shape[3] or block_table.dim() != 2):
        raise ValueError("expected q [B,q,H,D], k_pool and v_pool [rows,Hkv,D], block_table [B,max_blocks]")
    max_blocks = block_table.shape[1]
    _ints("block_table", block_table, q.shape[0], max_blocks)
    dev = q.get_device()
    if not (_on_current(dev) and dev == k_pool.get_device() == v_pool.get_device() == seq_lens.get_device()
            == tree_mask.get_device() == block_table.get_device()):
        _wrong_device(q, k_pool, v_pool, seq_lens, tree_mask, block_table)
    B, q_len, H, D, dt, strides, out, lse, ws = _gqa(q, k_pool, v_pool, seq_lens, tree_mask, out, lse, workspace, shape[1],
                                                     stream)
    if not dev == out.get_device() == lse.get_device() == ws.get_device():
        _wrong_device(q, out, lse, ws)
    st = _call(_GQA_PAGED, _pack_paged(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), strides and ctypes.addressof(strides), shape[0],
        block_table.data_ptr(), max_blocks, page_size, seq_lens.data_ptr(), tree_mask.data_ptr(), B, q_len, H, shape[1],
        D, dt, scale, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
        _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_verify_attn_paged")
    return out, lse


def gqa_verify_attn_window(q, k, v, seq_lens, tree_mask, scale, window, sinks=0, out=None, lse=None, workspace=None,
                           stream=None):
    """gqa_verify_attn with a sliding window: of the keys that its mask shows a
    draft, in the cache's order, it attends to the last ``window`` (>= 1) and to
    those in the cache's first ``sinks`` rows.  Rows from ``sinks`` up to
    seq_lens[b] - q - window are not used and may hold anything."""
    if _call is None:
        _bind()
    shape = k.shape
    if q.dim() != 4 or len(shape) != 4 or v.shape != shape or shape[0] != q.shape[0] or shape[3] != q.shape[3]:
        raise ValueError("expected q [B,q,H,D], k and v [B,Smax,Hkv,D]")
    dev = q.get_device()
    if not (_on_current(dev) and dev == k.get_device() == v.get_device() == seq_lens.get_device()
            == tree_mask.get_device()):
        _wrong_device(q, k, v, seq_lens, tree_mask)
    B, q_len, H, D, dt, strides, out, lse, ws = _gqa(q, k, v, seq_lens, tree_mask, out, lse, workspace, shape[2],
                                                     stream)
    if not dev == out.get_device() == lse.get_device() == ws.get_device():
        _wrong_device(q, out, lse, ws)
    st = _call(_WINDOW, _pack_window(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides and ctypes.addressof(strides), seq_lens.data_ptr(),
        tree_mask.data_ptr(), B, q_len, H, shape[2], D, shape[1], dt, scale, window, sinks, out.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_verify_attn_window")
    return out, lse


def gqa_verify_attn_window_paged(q, k_pool, v_pool, block_table, page_size, seq_lens, tree_mask, scale, window, sinks=0,
                                 out=None, lse=None, workspace=None, stream=None):
    """gqa_verify_attn_paged with a sliding window (see ``gqa_verify_attn_window``);
    table entries of pages that lie wholly between the first ``sinks`` rows and
    row seq_lens[b] - q - window are not read."""
    if _call is None:
        _bind()
    shape = k_pool.shape
    if (q.dim() != 4 or len(shape) != 3 or v_pool.shape != shape or shape[2] != q.shape[3] or block_table.dim() != 2):
        raise ValueError("expected q [B,q,H,D], k_pool and v_pool [rows,Hkv,D], block_table [B,max_blocks]")
    max_blocks = block_table.shape[1]
    _ints("block_table", block_table, q.shape[0], max_blocks)
    dev = q.get_device()
    if not (_on_current(dev) and dev == k_pool.get_device() == v_pool.get_device() == seq_lens.get_device()
            == tree_mask.get_device() == block_table.get_device()):
        _wrong_device(q, k_pool, v_pool, seq_lens, tree_mask, block_table)
    B, q_len, H, D, dt, strides, out, lse, ws = _gqa(q, k_pool, v_pool, seq_lens, tree_mask, out, lse, workspace,
                                                     shape[1], stream)
    if not dev == out.get_device() == lse.get_device() == ws.get_device():
        _wrong_device(q, out, lse, ws)
    st = _call(_WINDOW_PAGED, _pack_window_paged(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), strides and ctypes.addressof(strides), shape[0],
        block_table.data_ptr(), max_blocks, page_size, seq_lens.data_ptr(), tree_mask.data_ptr(), B, q_len, H, shape[1],
        D, dt, scale, window, sinks, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
        _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_verify_attn_window_paged")
    return out, lse


# ---------------------------------------------------------------- block tables

def blocks_extend(seq_lens, new_lens, block_table, page_size, free_pages, free_count, pool_pages, slots, stream=None):
    """Room for new_lens[b] tokens in every stream, in place: new blocks come off
    the stack free_pages[:free_count], seq_lens grows, and slots[t] becomes the
    pool row of the batch's t-th new token (-1 behind the last).

    All int32 and contiguous: seq_lens, new_lens [B], block_table
    [B,max_blocks], free_pages [n], free_count [1], slots [>= new tokens].
    Either the whole batch grows or nothing does (``last_device_error`` tells).
    """
    if _call is None:
        _bind()
    B, max_blocks, n_free, n_slots = (seq_lens.shape[0], block_table.shape[-1], free_pages.shape[0], slots.shape[0])
    i32 = _int32
    if not (seq_lens.dtype is i32 and new_lens.dtype is i32 and block_table.dtype is i32 and free_pages.dtype is i32
            and free_count.dtype is i32 and slots.dtype is i32 and seq_lens.dim() == 1 and new_lens.shape == (B,)
            and block_table.shape == (B, max_blocks) and free_pages.dim() == 1 and free_count.shape == (1,)
            and slots.dim() == 1 and seq_lens.is_contiguous() and new_lens.is_contiguous()
            and block_table.is_contiguous() and free_pages.is_contiguous() and slots.is_contiguous()):
        _wrong_ints(seq_lens=(seq_lens, B), new_lens=(new_lens, B), block_table=(block_table, B, max_blocks),
                    free_pages=(free_pages, n_free), free_count=(free_count, 1), slots=(slots, n_slots))
    dev = seq_lens.get_device()
    if not (_on_current(dev) and dev == new_lens.get_device() == block_table.get_device() == free_pages.get_device()
            == free_count.get_device() == slots.get_device()):
        _wrong_device(seq_lens, new_lens, block_table, free_pages, free_count, slots)
    st = _call(_EXTEND, _pack_extend(
        seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), B, max_blocks, page_size,
        free_pages.data_ptr(), n_free, free_count.data_ptr(), pool_pages, slots.data_ptr(), n_slots,
        _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_blocks_extend")


def blocks_trim(seq_lens, keep_lens, block_table, page_size, free_pages, free_count, stream=None):
    """Shortens every stream to keep_lens[b] tokens, in place, and puts the
    released pages back on the stack: the inverse of ``blocks_extend``."""
    if _call is None:
        _bind()
    B, max_blocks, n_free = seq_lens.shape[0], block_table.shape[-1], free_pages.shape[0]
    i32 = _int32
    if not (seq_lens.dtype is i32 and keep_lens.dtype is i32 and block_table.dtype is i32 and free_pages.dtype is i32
            and free_count.dtype is i32 and seq_lens.dim() == 1 and keep_lens.shape == (B,)
            and block_table.shape == (B, max_blocks) and free_pages.dim() == 1 and free_count.shape == (1,)
            and seq_lens.is_contiguous() and keep_lens.is_contiguous() and block_table.is_contiguous()
            and free_pages.is_contiguous()):
        _wrong_ints(seq_lens=(seq_lens, B), keep_lens=(keep_lens, B), block_table=(block_table, B, max_blocks),
                    free_pages=(free_pages, n_free), free_count=(free_count, 1))
    dev = seq_lens.get_device()
    if not (_on_current(dev) and dev == keep_lens.get_device() == block_table.get_device() == free_pages.get_device()
            == free_count.get_device()):
        _wrong_device(seq_lens, keep_lens, block_table, free_pages, free_count)
    st = _call(_TRIM, _pack_trim(
        seq_lens.data_ptr(), keep_lens.data_ptr(), block_table.data_ptr(), B, max_blocks, page_size,
        free_pages.data_ptr(), n_free, free_count.data_ptr(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_blocks_trim")


# ---------------------------------------------------------------- cache rows

def _rows(name, t, width):
    """Byte stride of bf16 rows [T, width] whose elements are contiguous."""
    shape, st = t.shape, t.stride()
    if t.dtype is not _bf16 or len(shape) != 2 or shape[1] != width or st[1] != 1:
        raise ValueError("%s must be bfloat16 [rows,%d] with contiguous rows" % (name, width))
    return 2 * st[0] if shape[0] > 1 else 2 * width


def _head_rows(name, t, dt, heads, width):
    """The same of rows [T, heads, width] of type dt."""
    shape, st = t.shape, t.stride()
    if (t.dtype is not dt or len(shape) != 3 or shape[1] != heads or shape[2] != width
            or (st[2] != 1 and width != 1) or (st[1] != width and heads != 1)):
        raise ValueError("%s must be [rows,%d,%d] of the pools' type with contiguous rows" % (name, heads, width))
    return 2 * st[0] if shape[0] > 1 else 2 * heads * width


def _pools(k_pool, v_pool):
    if k_pool.dim() != 3 or v_pool.shape != k_pool.shape:
        raise ValueError("expected k_pool and v_pool [rows,Hkv,D]")
    dt = k_pool.dtype
    if dt is not _bf16 and dt is not _fp16:
        raise ValueError("the pools must be bfloat16 or float16")
    rows, heads, width = k_pool.shape
    k_stride, v_stride = _head_rows("k_pool", k_pool, dt, heads, width), _head_rows("v_pool", v_pool, dt, heads, width)
    return dt, rows, heads, width, k_stride, v_stride


def cache_append(kv_pool, latent, rope, slots, stream=None):
    """Latent-cache rows by slot: kv_pool[slots[t]] = latent[t] (512) | rope[t] (64).

    kv_pool [rows,576], latent [T,512], rope [T,64], all bf16 (latent and rope
    may be column ranges of wider rows), slots [T] int32 as ``blocks_extend``
    makes them; a negative slot skips its token.
    """
    if _call is None:
        _bind()
    T = slots.shape[0]
    pool_stride = _rows("kv_pool", kv_pool, ROW)
    a_stride, b_stride = _rows("latent", latent, LATENT), _rows("rope", rope, ROPE)
    _ints("slots", slots, T)
    if latent.shape[0] != T or rope.shape[0] != T:
        raise ValueError("expected one slot a row")
    dev = kv_pool.get_device()
    if not (_on_current(dev) and dev == latent.get_device() == rope.get_device() == slots.get_device()):
        _wrong_device(kv_pool, latent, rope, slots)
    pool = kv_pool.data_ptr()
    st = _call(_APPEND, _pack_append(
        latent.data_ptr(), a_stride, 2 * LATENT, pool, pool_stride, rope.data_ptr(), b_stride, 2 * ROPE,
        pool + 2 * LATENT, pool_stride, kv_pool.shape[0], slots.data_ptr(), T, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_append")


def gqa_cache_append(k_pool, v_pool, k, v, slots, stream=None):
    """Key and value rows by slot: k_pool[slots[t]] = k[t], v_pool[slots[t]] = v[t];
    pools [rows,Hkv,D], k and v [T,Hkv,D] (column ranges of wider rows, too)."""
    if _call is None:
        _bind()
    T = slots.shape[0]
    dt, rows, heads, width, k_stride, v_stride = _pools(k_pool, v_pool)
    a_stride, b_stride = _head_rows("k", k, dt, heads, width), _head_rows("v", v, dt, heads, width)
    _ints("slots", slots, T)
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError("expected one slot a row")
    dev = k_pool.get_device()
    if not (_on_current(dev) and dev == v_pool.get_device() == k.get_device() == v.get_device() == slots.get_device()):
        _wrong_device(k_pool, v_pool, k, v, slots)
    n = 2 * heads * width
    st = _call(_APPEND, _pack_append(
        k.data_ptr(), a_stride, n, k_pool.data_ptr(), k_stride, v.data_ptr(), b_stride, n,
        v_pool.data_ptr(), v_stride, rows, slots.data_ptr(), T, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_append")


def _keep_tables(block_table, seq_lens, path, keep):
    if path.dim() != 2 or block_table.dim() != 2:
        raise ValueError("expected path [B,q] and block_table [B,max_blocks]")
    B, q_len = path.shape
    max_blocks = block_table.shape[1]
    i32 = _int32
    if not (path.dtype is i32 and keep.dtype is i32 and seq_lens.dtype is i32 and block_table.dtype is i32
            and keep.shape == (B,) and seq_lens.shape == (B,) and block_table.shape == (B, max_blocks)
            and path.is_contiguous() and keep.is_contiguous() and seq_lens.is_contiguous()
            and block_table.is_contiguous()):
        _wrong_ints(path=(path, B, q_len), keep=(keep, B), seq_lens=(seq_lens, B),
                    block_table=(block_table, B, max_blocks))
    return B, q_len, max_blocks


def cache_keep(kv_pool, block_table, page_size, seq_lens, path, keep, stream=None):
    """Moves the accepted drafts' rows together, in place: with prefix = seq_lens[b] - q,
    row prefix + j takes what row prefix + path[b,j] held, for j < keep[b].

    path [B,q] int32 draft indices, keep [B] int32; seq_lens stays as it is
    (``blocks_trim`` to prefix + keep follows).  A contiguous cache [B,Smax,576]
    is a pool of one page of Smax rows a stream.
    """
    if _call is None:
        _bind()
    pool_stride = _rows("kv_pool", kv_pool, ROW)
    B, q_len, max_blocks = _keep_tables(block_table, seq_lens, path, keep)
    dev = kv_pool.get_device()
    if not (_on_current(dev) and dev == block_table.get_device() == seq_lens.get_device() == path.get_device()
            == keep.get_device()):
        _wrong_device(kv_pool, block_table, seq_lens, path, keep)
    st = _call(_KEEP, _pack_keep(
        kv_pool.data_ptr(), pool_stride, 2 * ROW, 0, 0, 0, kv_pool.shape[0], block_table.data_ptr(),
        max_blocks, page_size, seq_lens.data_ptr(), path.data_ptr(), keep.data_ptr(), B, q_len, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_keep")


def gqa_cache_keep(k_pool, v_pool, block_table, page_size, seq_lens, path, keep, stream=None):
    """cache_keep for pools of separate keys and values [rows,Hkv,D]."""
    if _call is None:
        _bind()
    _, rows, heads, width, k_stride, v_stride = _pools(k_pool, v_pool)
    B, q_len, max_blocks = _keep_tables(block_table, seq_lens, path, keep)
    dev = k_pool.get_device()
    if not (_on_current(dev) and dev == v_pool.get_device() == block_table.get_device() == seq_lens.get_device()
            == path.get_device() == keep.get_device()):
        _wrong_device(k_pool, v_pool, block_table, seq_lens, path, keep)
    n = 2 * heads * width
    st = _call(_KEEP, _pack_keep(
        k_pool.data_ptr(), k_stride, n, v_pool.data_ptr(), v_stride, n, rows, block_table.data_ptr(),
        max_blocks, page_size, seq_lens.data_ptr(), path.data_ptr(), keep.data_ptr(), B, q_len, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_keep")


# ---------------------------------------------------------------- a cache in 4 bits

_row_bytes = {}


def gqa_fp4_row_bytes(Hkv: int, D: int) -> int:
    """Bytes of a pool row that holds Hkv heads of D = 64 or 128 values in 4 bits (0: not supported)."""
    n = _row_bytes.get((Hkv, D))
    if n is None:
        n = _row_bytes[Hkv, D] = int(load_library().mla_gqa_fp4_row_bytes(Hkv, D))
    return n


def _byte_rows(name, t, width):
    """Byte stride of uint8 rows [rows, width] whose bytes are contiguous."""
    shape, st = t.shape, t.stride()
    if t.dtype is not _uint8 or len(shape) != 2 or shape[1] != width or st[1] != 1:
        raise ValueError("%s must be uint8 [rows,%d] with contiguous rows" % (name, width))
    return st[0] if shape[0] > 1 else width


def _byte_pools(k_pool, v_pool):
    if k_pool.dim() != 2 or v_pool.shape != k_pool.shape:
        raise ValueError("expected k_pool and v_pool uint8 [rows,bytes]")
    rows, width = k_pool.shape
    return rows, width, _byte_rows("k_pool", k_pool, width), _byte_rows("v_pool", v_pool, width)


def gqa_cache_append_fp4(k_pool, v_pool, k, v, slots, k_scale=1.0, v_scale=1.0, k_held=None, v_held=None, stream=None):
    """Key and value rows by slot into pools held in 4 bits: uint8
    [rows, gqa_fp4_row_bytes(Hkv, D)], k and v [T,Hkv,D] bf16 or fp16 (column
    ranges of wider rows, too).

    Every 16 values share a step; k_scale and v_scale are the pools' own factors
    (a value is code * step * factor; steps reach from 2^-9 to 448).  With k_held,
    v_held [T,Hkv,D] of k's type, those take the values that the pools now hold.
    """
    if _call is None:
        _bind()
    shape, pool = k.shape, k_pool.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("expected k and v [T,Hkv,D]")
    T, heads, width = shape
    dt = k.dtype
    if dt is not _bf16 and dt is not _fp16:
        raise ValueError("k and v must be bfloat16 or float16")
    n = _row_bytes.get((heads, width)) or gqa_fp4_row_bytes(heads, width)
    ks, vs, kps, vps = k.stride(), v.stride(), k_pool.stride(), v_pool.stride()
    i32 = _int32
    # (Everything at once, and one by one where something is wrong.)
    if not (T > 1 and heads > 1 and ks[2] == 1 == vs[2] and ks[1] == width == vs[1] and v.dtype is dt and len(pool) == 2
            and pool == v_pool.shape and pool[1] == n and pool[0] > 1 and kps[1] == 1 == vps[1] and k_pool.dtype is _uint8
            and v_pool.dtype is _uint8 and slots.dtype is i32 and slots.shape == (T,) and slots.is_contiguous()):
        rows, n_bytes, k_pool_stride, v_pool_stride = _byte_pools(k_pool, v_pool)
        if n_bytes != n or n == 0:
            raise ValueError("k_pool and v_pool must be uint8 [rows,%d]" % n)
        k_stride, v_stride = _head_rows("k", k, dt, heads, width), _head_rows("v", v, dt, heads, width)
        _ints("slots", slots, T)
    else:
        rows, k_pool_stride, v_pool_stride, k_stride, v_stride = pool[0], kps[0], vps[0], 2 * ks[0], 2 * vs[0]
    dev = k_pool.get_device()
    if not (_on_current(dev) and dev == v_pool.get_device() == k.get_device() == v.get_device() == slots.get_device()):
        _wrong_device(k_pool, v_pool, k, v, slots)
    kh = vh = kh_stride = vh_stride = 0
    if k_held is not None:
        kh, kh_stride = _held("k_held", k_held, k, dev)
    if v_held is not None:
        vh, vh_stride = _held("v_held", v_held, k, dev)
    st = _call(_APPEND_FP4, _pack_append_fp4(
        k.data_ptr(), k_stride, v.data_ptr(), v_stride, heads, width, 0 if dt is _bf16 else 1, k_scale, v_scale,
        k_pool.data_ptr(), k_pool_stride, v_pool.data_ptr(), v_pool_stride, rows, slots.data_ptr(), T, kh, kh_stride, vh,
        vh_stride, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_cache_append_fp4")


def _held(name, t, like, dev):
    """Address and byte stride of rows of `like`'s shape and type that take held values."""
    if t.shape != like.shape:
        raise ValueError("%s must have k's shape" % name)
    if t.get_device() != dev:
        _wrong_device(like, t)
    if t.dtype is like.dtype and t.is_contiguous():
        return t.data_ptr(), 2 * t.shape[1] * t.shape[2]
    return t.data_ptr(), _head_rows(name, t, like.dtype, t.shape[1], t.shape[2])


def gqa_fp4_workspace_size(B: int, q_len: int, H: int, Hkv: int, D: int) -> int:
    """Workspace bytes of gqa_verify_attn_fp4_paged on the current device."""
    return int(load_library().mla_gqa_fp4_workspace_size(B, q_len, H, Hkv, D))


def gqa_verify_attn_fp4_paged(q, k_pool, v_pool, kv_heads, block_table, page_size, seq_lens, tree_mask, scale,
                              k_scale=1.0, v_scale=1.0, out=None, lse=None, workspace=None, stream=None):
    """gqa_verify_attn_paged over pools held in 4 bits, uint8
    [pool_rows, gqa_fp4_row_bytes(kv_heads, D)] as ``gqa_cache_append_fp4`` fills them
    with the same k_scale and v_scale; q [B,q,H,D] bf16 or fp16."""
    if _call is None:
        _bind()
    if q.dim() != 4 or block_table.dim() != 2:
        raise ValueError("expected q [B,q,H,D], block_table [B,max_blocks]")
    B, q_len, H, D = q.shape
    dt = q.dtype
    if dt is not _bf16 and dt is not _fp16:
        raise ValueError("q must be bfloat16 or float16")
    rows, width, k_stride, v_stride = _byte_pools(k_pool, v_pool)
    if width != gqa_fp4_row_bytes(kv_heads, D):
        raise ValueError("k_pool and v_pool must be uint8 [rows,%d]" % gqa_fp4_row_bytes(kv_heads, D))
    max_blocks = block_table.shape[1]
    _ints("block_table", block_table, B, max_blocks)
    _ints("seq_lens", seq_lens, B)
    if (tree_mask.element_size() != 4 or tree_mask.shape != (B, q_len, (q_len + 31) >> 5)
            or not tree_mask.is_contiguous() or tree_mask.is_floating_point()):
        raise ValueError("tree_mask must be contiguous 32-bit words [B,q,ceil(q/32)]")
    dev = q.get_device()
    if not (_on_current(dev) and dev == k_pool.get_device() == v_pool.get_device() == seq_lens.get_device()
            == tree_mask.get_device() == block_table.get_device()):
        _wrong_device(q, k_pool, v_pool, seq_lens, tree_mask, block_table)
    strides = 0
    if not q.is_contiguous():
        qs = q.stride()
        if qs[3] != 1:
            raise ValueError("the innermost dimension of q must be contiguous")
        strides = _STRIDES(*qs[:3], 0, 0, 0, 0, 0, 0)
    if out is None:
        out = _empty((B, q_len, H, D), dt, q, stream)
    elif out.dtype is not dt or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is None:
        lse = _empty((B, q_len, H), _fp32, q, stream)
    elif lse.dtype is not _fp32 or lse.shape != (B, q_len, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,q,H]")
    if workspace is None:
        workspace = _empty(gqa_fp4_workspace_size(B, q_len, H, kv_heads, D), _uint8, q, stream, result=False)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not dev == out.get_device() == lse.get_device() == workspace.get_device():
        _wrong_device(q, out, lse, workspace)
    st = _call(_FP4_PAGED, _pack_fp4_paged(
        q.data_ptr(), strides and ctypes.addressof(strides), k_pool.data_ptr(), k_stride, v_pool.data_ptr(), v_stride,
        rows, block_table.data_ptr(), max_blocks, page_size, seq_lens.data_ptr(), tree_mask.data_ptr(), B, q_len, H,
        kv_heads, D, 0 if dt is _bf16 else 1, scale, k_scale, v_scale, out.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_verify_attn_fp4_paged")
    return out, lse


def gqa_cache_keep_fp4(k_pool, v_pool, block_table, page_size, seq_lens, path, keep, stream=None):
    """gqa_cache_keep for pools held in 4 bits, uint8 [rows,bytes]."""
    if _call is None:
        _bind()
    rows, n, k_stride, v_stride = _byte_pools(k_pool, v_pool)
    B, q_len, max_blocks = _keep_tables(block_table, seq_lens, path, keep)
    dev = k_pool.get_device()
    if not (_on_current(dev) and dev == v_pool.get_device() == block_table.get_device() == seq_lens.get_device()
            == path.get_device() == keep.get_device()):
        _wrong_device(k_pool, v_pool, block_table, seq_lens, path, keep)
    st = _call(_KEEP, _pack_keep(
        k_pool.data_ptr(), k_stride, n, v_pool.data_ptr(), v_stride, n, rows, block_table.data_ptr(),
        max_blocks, page_size, seq_lens.data_ptr(), path.data_ptr(), keep.data_ptr(), B, q_len, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_keep")


# ---------------------------------------------------------------- eviction

def evict_workspace_size(B: int, Smax: int) -> int:
    """Workspace bytes of evict_select (0 for streams of up to 393,216 keys)."""
    return int(load_library().mla_evict_workspace_size(B, Smax))


def _weights(q, k, seq_lens, tree_mask, lse, weights, Hkv, Smax):
    B, q_len, H, D = q.shape
    dt = q.dtype
    if k.dtype is not dt or (dt is not _bf16 and dt is not _fp16):
        raise ValueError("q and k must have one type, bfloat16 or float16")
    _ints("seq_lens", seq_lens, B)
    if (tree_mask.element_size() != 4 or tree_mask.shape != (B, q_len, (q_len + 31) >> 5)
            or not tree_mask.is_contiguous() or tree_mask.is_floating_point()):
        raise ValueError("tree_mask must be contiguous 32-bit words [B,q,ceil(q/32)]")
    if lse.dtype is not _fp32 or lse.shape != (B, q_len, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,q,H]")
    if weights.dtype is not _fp32 or weights.shape != (B, Hkv, Smax) or not weights.is_contiguous():
        raise ValueError("weights must be contiguous float32 [B,Hkv,%d]" % Smax)
    strides = 0
    if not (q.is_contiguous() and k.is_contiguous()):
        qs, ks = q.stride(), k.stride()
        if qs[3] != 1 or ks[-1] != 1:
            raise ValueError("the innermost dimension of q and k must be contiguous")
        if len(ks) == 3:            # pools: no batch dimension
            ks = (8,) + ks
        strides = _STRIDES(*qs[:3], *ks[:3], 0, 0, 0)
    return B, q_len, H, D, 0 if dt is _bf16 else 1, strides


def gqa_attn_weights(q, k, seq_lens, tree_mask, lse, scale, weights, stream=None):
    """Adds the attention weight that each cached key got, in place: weights[b,g,t]
    += sum of exp(score - lse) over the drafts that see key t and the query heads of
    key head g.

    q, k, seq_lens and tree_mask as for ``gqa_verify_attn``, lse [B,q,H] as it
    returns it (rows with lse +inf or -inf add nothing: +inf leaves out drafts
    that were not accepted), weights [B,Hkv,Smax] fp32.

    Sums belong to places of the cache: ``gqa_cache_keep`` moves the accepted
    drafts' rows without their sums, ``blocks_trim`` leaves those of the places that
    it gives up.  Move them along and clear what is behind them, or use
    ``gqa_cache_compact`` with weights in place of ``gqa_cache_keep``.
    """
    if _call is None:
        _bind()
    shape = k.shape
    if q.dim() != 4 or len(shape) != 4 or shape[0] != q.shape[0] or shape[3] != q.shape[3]:
        raise ValueError("expected q [B,q,H,D], k [B,Smax,Hkv,D]")
    dev = q.get_device()
    if not (_on_current(dev) and dev == k.get_device() == seq_lens.get_device() == tree_mask.get_device()
            == lse.get_device() == weights.get_device()):
        _wrong_device(q, k, seq_lens, tree_mask, lse, weights)
    B, q_len, H, D, dt, strides = _weights(q, k, seq_lens, tree_mask, lse, weights, shape[2], shape[1])
    st = _call(_WEIGHTS, _pack_weights(
        q.data_ptr(), k.data_ptr(), strides and ctypes.addressof(strides), seq_lens.data_ptr(), tree_mask.data_ptr(),
        lse.data_ptr(), B, q_len, H, shape[2], D, shape[1], dt, scale, weights.data_ptr(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_attn_weights")


def gqa_attn_weights_paged(q, k_pool, block_table, page_size, seq_lens, tree_mask, lse, scale, weights, stream=None):
    """gqa_attn_weights over a pool k_pool [pool_rows,Hkv,D] of pages of page_size >= 1
    rows, block_table [B,max_blocks] int32, weights [B,Hkv,max_blocks * page_size]."""
    if _call is None:
        _bind()
    shape = k_pool.shape
    if q.dim() != 4 or len(shape) != 3 or shape[2] != q.shape[3] or block_table.dim() != 2:
        raise ValueError("expected q [B,q,H,D], k_pool [rows,Hkv,D], block_table [B,max_blocks]")
    max_blocks = block_table.shape[1]
    _ints("block_table", block_table, q.shape[0], max_blocks)
    dev = q.get_device()
    if not (_on_current(dev) and dev == k_pool.get_device() == seq_lens.get_device() == tree_mask.get_device()
            == block_table.get_device() == lse.get_device() == weights.get_device()):
        _wrong_device(q, k_pool, seq_lens, tree_mask, block_table, lse, weights)
    B, q_len, H, D, dt, strides = _weights(q, k_pool, seq_lens, tree_mask, lse, weights, shape[1], max_blocks * page_size)
    st = _call(_WEIGHTS_PAGED, _pack_weights_paged(
        q.data_ptr(), k_pool.data_ptr(), strides and ctypes.addressof(strides), shape[0], block_table.data_ptr(),
        max_blocks, page_size, seq_lens.data_ptr(), tree_mask.data_ptr(), lse.data_ptr(), B, q_len, H, shape[1], D, dt,
        scale, weights.data_ptr(), _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_gqa_attn_weights_paged")


def evict_select(weights, seq_lens, sinks, recent, kept, keep_lens, workspace=None, stream=None):
    """Which keys of each stream stay: the first ``sinks``, the last ``recent`` and,
    to kept.shape[1] in all, those between with the largest sums of weights over
    the heads (of equal ones the first).

    weights [B,Hkv,Smax] fp32 as ``gqa_attn_weights`` adds them up, seq_lens [B].
    Writes kept [B,budget] (positions in order, -1 behind them) and keep_lens [B],
    both int32: ``gqa_cache_compact`` and ``blocks_trim`` to keep_lens follow.
    """
    if _call is None:
        _bind()
    if weights.dim() != 3 or weights.dtype is not _fp32 or not weights.is_contiguous():
        raise ValueError("weights must be contiguous float32 [B,Hkv,Smax]")
    B, heads, Smax = weights.shape
    budget = kept.shape[-1]
    _ints("seq_lens", seq_lens, B)
    _ints("kept", kept, B, budget)
    _ints("keep_lens", keep_lens, B)
    dev = weights.get_device()
    if not (_on_current(dev) and dev == seq_lens.get_device() == kept.get_device() == keep_lens.get_device()):
        _wrong_device(weights, seq_lens, kept, keep_lens)
    at = size = 0
    if workspace is None and Smax > 49152:           # (shorter streams need none)
        n = evict_workspace_size(B, Smax)
        workspace = _empty(n, _uint8, weights, stream, result=False) if n else None
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.get_device() != dev:
            _wrong_device(weights, workspace)
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _call(_SELECT, _pack_select(
        weights.data_ptr(), seq_lens.data_ptr(), B, heads, Smax, sinks, recent, kept.data_ptr(), budget,
        keep_lens.data_ptr(), at, size, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_evict_select")


def _compact(pool_a, a_stride, a_bytes, pool_b, b_stride, b_bytes, rows, weights, block_table, page_size, seq_lens, kept,
             keep_lens, stream):
    if block_table.dim() != 2 or kept.dim() != 2:
        raise ValueError("expected block_table [B,max_blocks] and kept [B,budget]")
    B, max_blocks = block_table.shape
    budget = kept.shape[1]
    _ints("block_table", block_table, B, max_blocks)
    _ints("seq_lens", seq_lens, B)
    _ints("kept", kept, B, budget)
    _ints("keep_lens", keep_lens, B)
    w = heads = 0
    dev = pool_a.get_device()
    if not (_on_current(dev) and dev == pool_b.get_device() == block_table.get_device() == seq_lens.get_device()
            == kept.get_device() == keep_lens.get_device()):
        _wrong_device(pool_a, pool_b, block_table, seq_lens, kept, keep_lens)
    if weights is not None:
        heads = weights.shape[1] if weights.dim() == 3 else 0
        if (weights.dtype is not _fp32 or weights.shape != (B, heads, max_blocks * page_size)
                or not weights.is_contiguous()):
            raise ValueError("weights must be contiguous float32 [B,Hkv,max_blocks * page_size]")
        if weights.get_device() != dev:
            _wrong_device(pool_a, weights)
        w = weights.data_ptr()
    st = _call(_COMPACT, _pack_compact(
        pool_a.data_ptr(), a_stride, a_bytes, pool_b.data_ptr() if b_bytes else 0, b_stride, b_bytes, rows, w, heads,
        block_table.data_ptr(), max_blocks, page_size, seq_lens.data_ptr(), kept.data_ptr(), budget,
        keep_lens.data_ptr(), B, _handle(stream, dev)))
    if st != MLA_OK:
        raise MLAError(st, "mla_cache_compact")


def gqa_cache_compact(k_pool, v_pool, block_table, page_size, seq_lens, kept, keep_lens, weights=None, stream=None):
    """Moves the rows that stay together, in place: row j of stream b takes what row
    kept[b,j] held, for j < keep_lens[b] (both as ``evict_select`` leaves them).

    Pools [rows,Hkv,D] bf16 or fp16, or uint8 [rows,bytes] held in 4 bits; weights
    [B,Hkv,max_blocks * page_size] move along, with zeros behind.  seq_lens stays
    as it is (``blocks_trim`` to keep_lens follows).
    """
    if _call is None:
        _bind()
    if k_pool.dtype is _uint8:
        rows, n, k_stride, v_stride = _byte_pools(k_pool, v_pool)
    else:
        _, rows, heads, width, k_stride, v_stride = _pools(k_pool, v_pool)
        n = 2 * heads * width
    _compact(k_pool, k_stride, n, v_pool, v_stride, n, rows, weights, block_table, page_size, seq_lens, kept, keep_lens,
             stream)


def cache_compact(kv_pool, block_table, page_size, seq_lens, kept, keep_lens, weights=None, stream=None):
    """gqa_cache_compact for a latent pool [rows,576] bf16."""
    if _call is None:
        _bind()
    stride = _rows("kv_pool", kv_pool, ROW)
    _compact(kv_pool, stride, 2 * ROW, kv_pool, 0, 0, kv_pool.shape[0], weights, block_table, page_size, seq_lens, kept,
             keep_lens, stream)
