"""Bindings of the grouped-head verify attention and of the cache operators.

Argument marshalling only, as in ``_lib``: shapes, types and devices are
checked, addresses and strides passed on, and a status other than MLA_OK
raises ``MLAError``.  Problems only the GPU can see are in
``last_device_error``.
"""
from __future__ import annotations

import ctypes

from ._lib import MLA_OK, MLAError, load_library

_fn = {}
_STRIDES = ctypes.c_longlong * 9


def _f(name):
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(load_library(), name)
    return f


def _dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise ValueError("expected bfloat16 or float16 tensors, got %s" % t.dtype)


def _device(tensors):
    """The tensors' device index: one CUDA device, the current one."""
    import torch
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if dev != torch.cuda.current_device():
        raise ValueError("the tensors' device must be the current one")
    return dev


def _handle(stream, dev, scratch=()):
    """The stream's handle; memory made here for another stream than the
    current one is recorded on it, so that it is not handed out too early."""
    import torch
    current = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return current
    handle = int(stream.cuda_stream)
    if handle != current:
        for t in scratch:
            t.record_stream(stream)
    return handle


def _ints(name, t, shape):
    import torch
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s" % (name, list(shape)))


def _check(st, what):
    if st != MLA_OK:
        raise MLAError(st, what)


# ---------------------------------------------------------------- attention

def gqa_workspace_size(B: int, q_len: int, H: int, Hkv: int, D: int) -> int:
    """Workspace bytes of the two calls below on the current device."""
    return int(_f("mla_gqa_workspace_size")(B, q_len, H, Hkv, D))


def _gqa(q, k, v, seq_lens, tree_mask, out, lse, workspace, Hkv, others):
    import torch
    B, q_len, H, D = q.shape
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one type")
    dt = _dtype(q)
    _ints("seq_lens", seq_lens, (B,))
    if (tree_mask.element_size() != 4 or tree_mask.is_floating_point() or not tree_mask.is_contiguous()
            or tree_mask.shape != (B, q_len, (q_len + 31) >> 5)):
        raise ValueError("tree_mask must be contiguous 32-bit words [B,q,ceil(q/32)]")
    if q.stride(3) != 1 or k.stride(-1) != 1 or v.stride(-1) != 1:
        raise ValueError("the innermost dimension of q, k and v must be contiguous")
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        ks, vs = k.stride(), v.stride()
        if len(ks) == 3:            # pools: no batch dimension
            ks, vs = (8,) + ks, (8,) + vs
        strides = _STRIDES(*q.stride()[:3], *ks[:3], *vs[:3])
    tensors = [q, k, v, seq_lens, tree_mask, *others]
    made = []
    if out is None:
        out = torch.empty((B, q_len, H, D), dtype=q.dtype, device=q.device)
        made.append(out)
    elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is None:
        lse = torch.empty((B, q_len, H), dtype=torch.float32, device=q.device)
        made.append(lse)
    elif lse.dtype != torch.float32 or lse.shape != (B, q_len, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,q,H]")
    if workspace is None:
        workspace = torch.empty(gqa_workspace_size(B, q_len, H, Hkv, D), dtype=torch.uint8, device=q.device)
        made.append(workspace)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    tensors += [out, lse, workspace]
    return dt, strides, out, lse, workspace, _device(tensors), made


def gqa_verify_attn(q, k, v, seq_lens, tree_mask, scale, out=None, lse=None, workspace=None, stream=None):
    """Verify attention with grouped query heads on the current CUDA device.

    q [B,q,H,D], k and v [B,Smax,Hkv,D], bf16 or fp16, D 64 or 128, H a
    multiple of Hkv; strided views are taken as they are if the innermost
    dimension is contiguous.  seq_lens [B] int32 counts the drafts' own rows
    (0: unused stream), tree_mask [B,q,ceil(q/32)] as for ``verify_attn``.
    Returns (out [B,q,H,D] in q's type, lse [B,q,H] fp32); a row whose mask
    leaves nothing has out 0 and lse -inf.
    """
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ValueError("expected q [B,q,H,D], k and v [B,Smax,Hkv,D]")
    B, q_len, H, D = q.shape
    Smax, Hkv = k.shape[1], k.shape[2]
    dt, strides, out, lse, ws, dev, made = _gqa(q, k, v, seq_lens, tree_mask, out, lse, workspace, Hkv, ())
    _check(_f("mla_gqa_verify_attn")(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, seq_lens.data_ptr(), tree_mask.data_ptr(), B, q_len, H,
        Hkv, D, Smax, dt, scale, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
        _handle(stream, dev, made)), "mla_gqa_verify_attn")
    return out, lse


def gqa_verify_attn_paged(q, k_pool, v_pool, block_table, page_size, seq_lens, tree_mask, scale, out=None, lse=None,
                          workspace=None, stream=None):
    """gqa_verify_attn over pools k_pool, v_pool [pool_rows,Hkv,D] of pages of
    page_size >= 1 rows, block_table [B,max_blocks] int32; read in place."""
    if (q.dim() != 4 or k_pool.dim() != 3 or v_pool.shape != k_pool.shape or k_pool.shape[2] != q.shape[3]
            or block_table.dim() != 2):
        raise ValueError("expected q [B,q,H,D], k_pool and v_pool [rows,Hkv,D], block_table [B,max_blocks]")
    B, q_len, H, D = q.shape
    rows, Hkv = k_pool.shape[0], k_pool.shape[1]
    _ints("block_table", block_table, (B, block_table.shape[1]))
    dt, strides, out, lse, ws, dev, made = _gqa(q, k_pool, v_pool, seq_lens, tree_mask, out, lse, workspace, Hkv,
                                                (block_table,))
    _check(_f("mla_gqa_verify_attn_paged")(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), strides, rows, block_table.data_ptr(),
        block_table.shape[1], page_size, seq_lens.data_ptr(), tree_mask.data_ptr(), B, q_len, H, Hkv, D, dt, scale,
        out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), _handle(stream, dev, made)),
        "mla_gqa_verify_attn_paged")
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
    B = seq_lens.shape[0]
    _ints("seq_lens", seq_lens, (B,))
    _ints("new_lens", new_lens, (B,))
    _ints("block_table", block_table, (B, block_table.shape[-1]))
    _ints("free_pages", free_pages, (free_pages.shape[0],))
    _ints("free_count", free_count, (1,))
    _ints("slots", slots, (slots.shape[0],))
    dev = _device((seq_lens, new_lens, block_table, free_pages, free_count, slots))
    _check(_f("mla_blocks_extend")(
        seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), B, block_table.shape[1], page_size,
        free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), pool_pages, slots.data_ptr(),
        slots.shape[0], _handle(stream, dev)), "mla_blocks_extend")


def blocks_trim(seq_lens, keep_lens, block_table, page_size, free_pages, free_count, stream=None):
    """Shortens every stream to keep_lens[b] tokens, in place, and puts the
    released pages back on the stack: the inverse of ``blocks_extend``."""
    B = seq_lens.shape[0]
    _ints("seq_lens", seq_lens, (B,))
    _ints("keep_lens", keep_lens, (B,))
    _ints("block_table", block_table, (B, block_table.shape[-1]))
    _ints("free_pages", free_pages, (free_pages.shape[0],))
    _ints("free_count", free_count, (1,))
    dev = _device((seq_lens, keep_lens, block_table, free_pages, free_count))
    _check(_f("mla_blocks_trim")(
        seq_lens.data_ptr(), keep_lens.data_ptr(), block_table.data_ptr(), B, block_table.shape[1], page_size,
        free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), _handle(stream, dev)), "mla_blocks_trim")


# ---------------------------------------------------------------- cache rows

LATENT, ROW = 512, 576


def _row_bytes(name, t, row_shape):
    """Row stride of [T, ...] rows whose inner dimensions are contiguous, in bytes."""
    want = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != want:
            raise ValueError("the rows of %s must be contiguous" % name)
        want *= n
    if tuple(t.shape[1:]) != tuple(row_shape):
        raise ValueError("%s must have rows of shape %s" % (name, list(row_shape)))
    size = want * t.element_size()
    return (t.stride(0) * t.element_size() if t.shape[0] > 1 else size), size


def _append(what, pool_a, pool_a_ptr, pool_a_stride, a, a_stride, a_bytes, pool_b, pool_b_ptr, pool_b_stride, b,
            b_stride, b_bytes, slots, stream):
    T = slots.shape[0]
    _ints("slots", slots, (T,))
    if a.shape[0] != T or b.shape[0] != T:
        raise ValueError("expected one slot a row")
    dev = _device((pool_a, pool_b, a, b, slots))
    _check(_f("mla_cache_append")(
        a.data_ptr(), a_stride, a_bytes, pool_a_ptr, pool_a_stride, b.data_ptr(), b_stride, b_bytes, pool_b_ptr,
        pool_b_stride, pool_a.shape[0], slots.data_ptr(), T, _handle(stream, dev)), what)


def _latent_pool(kv_pool):
    import torch
    if kv_pool.dim() != 2 or kv_pool.dtype != torch.bfloat16:
        raise ValueError("expected kv_pool [rows,576] bfloat16")
    stride, _ = _row_bytes("kv_pool", kv_pool, (ROW,))
    return kv_pool.data_ptr(), stride


def _pools(k_pool, v_pool):
    if k_pool.dim() != 3 or v_pool.shape != k_pool.shape or v_pool.dtype != k_pool.dtype:
        raise ValueError("expected k_pool and v_pool [rows,Hkv,D] of one type")
    _dtype(k_pool)
    row = k_pool.shape[1:]
    return row, _row_bytes("k_pool", k_pool, row), _row_bytes("v_pool", v_pool, row)


def cache_append(kv_pool, latent, rope, slots, stream=None):
    """Latent-cache rows by slot: kv_pool[slots[t]] = latent[t] (512) | rope[t] (64).

    kv_pool [rows,576], latent [T,512], rope [T,64], all bf16 (latent and rope
    may be column ranges of wider rows), slots [T] int32 as ``blocks_extend``
    makes them; a negative slot skips its token.
    """
    ptr, stride = _latent_pool(kv_pool)
    if latent.dtype != kv_pool.dtype or rope.dtype != kv_pool.dtype:
        raise ValueError("latent and rope must be bfloat16")
    (sa, na), (sb, nb) = _row_bytes("latent", latent, (LATENT,)), _row_bytes("rope", rope, (ROW - LATENT,))
    _append("mla_cache_append", kv_pool, ptr, stride, latent, sa, na, kv_pool, ptr + 2 * LATENT, stride, rope, sb, nb,
            slots, stream)


def gqa_cache_append(k_pool, v_pool, k, v, slots, stream=None):
    """Key and value rows by slot: k_pool[slots[t]] = k[t], v_pool[slots[t]] = v[t];
    pools [rows,Hkv,D], k and v [T,Hkv,D] (column ranges of wider rows, too)."""
    row, (ka, _), (va, _) = _pools(k_pool, v_pool)
    if k.dtype != k_pool.dtype or v.dtype != k_pool.dtype:
        raise ValueError("k and v must have the pools' type")
    (sk, nk), (sv, nv) = _row_bytes("k", k, row), _row_bytes("v", v, row)
    _append("mla_cache_append", k_pool, k_pool.data_ptr(), ka, k, sk, nk, v_pool, v_pool.data_ptr(), va, v, sv, nv,
            slots, stream)


def _keep(pool_a, ptr_a, stride_a, bytes_a, pool_b, ptr_b, stride_b, bytes_b, block_table, page_size, seq_lens, path,
          keep, stream):
    if path.dim() != 2 or block_table.dim() != 2:
        raise ValueError("expected path [B,q] and block_table [B,max_blocks]")
    B, q_len = path.shape
    _ints("path", path, (B, q_len))
    _ints("keep", keep, (B,))
    _ints("seq_lens", seq_lens, (B,))
    _ints("block_table", block_table, (B, block_table.shape[1]))
    dev = _device((pool_a, pool_b, block_table, seq_lens, path, keep))
    _check(_f("mla_cache_keep")(
        ptr_a, stride_a, bytes_a, ptr_b, stride_b, bytes_b, pool_a.shape[0], block_table.data_ptr(),
        block_table.shape[1], page_size, seq_lens.data_ptr(), path.data_ptr(), keep.data_ptr(), B, q_len,
        _handle(stream, dev)), "mla_cache_keep")


def cache_keep(kv_pool, block_table, page_size, seq_lens, path, keep, stream=None):
    """Moves the accepted drafts' rows together, in place: with prefix = seq_lens[b] - q,
    row prefix + j takes what row prefix + path[b,j] held, for j < keep[b].

    path [B,q] int32 draft indices, keep [B] int32; seq_lens stays as it is
    (``blocks_trim`` to prefix + keep follows).  A contiguous cache [B,Smax,576]
    is a pool of one page of Smax rows a stream.
    """
    ptr, stride = _latent_pool(kv_pool)
    _keep(kv_pool, ptr, stride, 2 * ROW, kv_pool, 0, 0, 0, block_table, page_size, seq_lens, path, keep, stream)


def gqa_cache_keep(k_pool, v_pool, block_table, page_size, seq_lens, path, keep, stream=None):
    """cache_keep for pools of separate keys and values [rows,Hkv,D]."""
    _, (sk, nk), (sv, nv) = _pools(k_pool, v_pool)
    _keep(k_pool, k_pool.data_ptr(), sk, nk, v_pool, v_pool.data_ptr(), sv, nv, block_table, page_size, seq_lens,
          path, keep, stream)
