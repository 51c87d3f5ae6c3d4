"""Plain 64-bit forms of the grouped-head verify attention, and the bounds its
results are held to."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def mask_words(seen):
    """[B,q,q] truth values (draft i sees draft j) -> int32 words [B,q,ceil(q/32)]."""
    B, q, _ = seen.shape
    words = -(-q // 32)
    bits = torch.zeros((B, q, words * 32), dtype=torch.int64)
    bits[:, :, :q] = seen.long()
    w = (bits.view(B, q, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def attend(q, k, v, n, seen, scale):
    """One stream in 64 bits: q [q,H,D], k and v [>=n,Hkv,D], n keys, seen [q,q].
    Returns out [q,H,D], lse [q,H], and the bound of out's error (see below)."""
    qn, H, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    dt = q.dtype
    if n == 0:
        z = torch.zeros((qn, H, D), dtype=torch.float64, device=q.device)
        return z, torch.full((qn, H), -float("inf"), dtype=torch.float64, device=q.device), z, z[..., 0]
    k, v = k[:n].double(), v[:n].double()
    see = torch.ones((qn, n), dtype=torch.bool, device=q.device)
    see[:, n - qn:] = seen.to(q.device)
    qd = q.double().view(qn, Hkv, G, D)
    s = torch.einsum("ihgd,thd->ihgt", qd, k) * scale
    size = torch.einsum("ihgd,thd->ihgt", qd.abs(), k.abs()) * abs(scale)
    hidden = ~see[:, None, None, :].expand_as(s)
    s = s.masked_fill(hidden, -float("inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = (s - top).exp()
    l = w.sum(-1, keepdim=True)
    safe = torch.where(l > 0, l, torch.ones_like(l))
    w = w / safe
    out = torch.einsum("ihgt,thd->ihgd", w, v)
    lse = torch.where(l > 0, top + safe.log(), torch.full_like(l, -float("inf")))[..., 0]
    # Error of a score: D products and sums in fp32 (D + 2 roundings of 2^-24 of
    # the sum of magnitudes), its scaling, and ex2's 2^-22: a relative error e of
    # every weight, twice (product and normaliser).  Each weight is rounded to
    # the type (u), the result once more (u); fp32 accumulation over n keys adds
    # n roundings of 2^-24 at worst.  fp16 weights below 2^-32 of the row's
    # largest are rounded to that step.
    e = (D + 4) * 2.0 ** -24 * size.masked_fill(hidden, 0).amax(-1) + 2.0 ** -21
    mass = torch.einsum("ihgt,thd->ihgd", w, v.abs())
    u = U[dt]
    bound = u * out.abs() + (u + 2 * e[..., None] + n * 2.0 ** -24) * mass * 1.01 + n * 2.0 ** -32 * v.abs().amax()
    # out below the type's normal range is rounded to a fixed step.
    bound = bound + (2.0 ** -25 if dt == torch.float16 else 0.0)
    lse_bound = e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + lse.abs().nan_to_num(posinf=0.0))
    return out.reshape(qn, H, D), lse.reshape(qn, H), bound.reshape(qn, H, D), lse_bound.reshape(qn, H)


def check(got_out, got_lse, q, k_of, v_of, lens, seen, scale):
    """Every stream's results against 64 bits; k_of(b), v_of(b) give its rows."""
    for b, n in enumerate(lens):
        out, lse, bound, lse_bound = attend(q[b], k_of(b), v_of(b), n, seen[b], scale)
        o, l = got_out[b].double(), got_lse[b].double()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isneginf(l), empty), "stream %d: empty rows" % b
        assert torch.isfinite(o).all(), "stream %d: not finite" % b
        off = (o - out).abs()
        assert (off <= bound).all(), "stream %d: off by %.3g, %.3g times its bound" % (
            b, off.max().item(), (off / bound.clamp_min(1e-300)).max().item())
        d = (l - lse).abs()[~empty]
        assert (d <= lse_bound[~empty]).all(), "stream %d: lse off by %.3g" % (b, d.max().item())
