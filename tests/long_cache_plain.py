"""Plain 64-bit forms of the operators that keep a long cache small, and the
bounds their results are held to."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def seen_keys(seen, n, window=None, sinks=0):
    """[q,n]: what each draft attends to of n keys, the last q of them the drafts (seen [q,q])."""
    q = seen.shape[0]
    see = torch.ones((q, n), dtype=torch.bool)
    see[:, n - q:] = seen
    if window is not None:
        for i in range(q):
            at = see[i].nonzero()[:, 0]
            see[i] = False
            see[i, at[max(len(at) - window, 0):]] = True
            see[i, at[at < sinks]] = True
    return see


def attend(q, k, v, see, scale, weight_u=None):
    """One stream in 64 bits: q [q,H,D], k and v [n,Hkv,D], see [q,n].  Returns out [q,H,D],
    lse [q,H] and the bounds of their errors.  weight_u: half a step of the weights' type (default: q's)."""
    qn, H, D = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    G = H // Hkv
    dt = q.dtype
    used = see.any(0).to(q.device)
    k, v = (torch.where(used[:, None, None], x.double(), 0.0) for x in (k, v))   # the others may hold anything
    see = see.to(q.device)
    qd = q.double().view(qn, Hkv, G, D)
    s = torch.einsum("ihgd,thd->ihgt", qd, k) * scale
    size = torch.einsum("ihgd,thd->ihgt", qd.abs(), k.abs()) * abs(scale)
    hidden = ~see[:, None, None, :].expand_as(s)
    s = s.masked_fill(hidden, -float("inf"))
    top = s.amax(-1, keepdim=True) if n else torch.full((qn, Hkv, G, 1), -float("inf"), device=q.device).double()
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
    # its type (wu), the result once (u); fp32 accumulation over n keys adds n
    # roundings of 2^-24 at worst.  fp16 weights below 2^-32 of the row's largest
    # are rounded to that step.
    e = (D + 4) * 2.0 ** -24 * size.masked_fill(hidden, 0).amax(-1) + 2.0 ** -21 if n else torch.zeros_like(lse)
    mass = torch.einsum("ihgt,thd->ihgd", w, v.abs())
    u = U[dt]
    wu = u if weight_u is None else weight_u
    m = int(see.sum(-1).max()) if n else 0
    most = v.abs().amax() if n else 0.0
    bound = u * out.abs() + (wu + 2 * e[..., None] + m * 2.0 ** -24) * mass * 1.01 + m * 2.0 ** -32 * most
    # out below the type's normal range is rounded to a fixed step.
    bound = bound + (2.0 ** -25 if dt == torch.float16 else 0.0)
    lse_bound = e + m * 2.0 ** -24 + 2.0 ** -22 * (1 + lse.abs().nan_to_num(posinf=0.0))
    return out.reshape(qn, H, D), lse.reshape(qn, H), bound.reshape(qn, H, D), lse_bound.reshape(qn, H)


def check(got_out, got_lse, want, name=""):
    """One stream's results against what `attend` gives."""
    out, lse, bound, lse_bound = want
    o, l = got_out.double(), got_lse.double()
    empty = torch.isinf(lse)
    assert torch.equal(torch.isneginf(l), empty), "%s: empty rows" % name
    assert torch.isfinite(o).all(), "%s: not finite" % name
    off = (o - out).abs()
    assert (off <= bound).all(), "%s: off by %.3g, %.3g times its bound" % (
        name, off.max().item(), (off / bound.clamp_min(1e-300)).max().item())
    d = (l - lse).abs()[~empty]
    assert (d <= lse_bound[~empty]).all(), "%s: lse off by %.3g" % (name, d.max().item())


def pages(gen, lens, page, spare=3):
    """A block table over a pool of pages in random order: (table [B,n], pages)."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(counts), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def rows_of(table_row, page, n):
    """Pool rows of a stream's first n keys."""
    t = torch.arange(n)
    return (table_row.cpu().long()[t // page] * page + t % page).clamp_min(0)


# ---------------------------------------------------------------- rows in 4 bits

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_values():
    """The 8-bit type's values by code, 0 .. 126, in 64 bits."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)],
                        dtype=torch.float64)


def nearest_even(x, values):
    """Index of the nearest of rising values, of two as near the even index; beyond the last, the last."""
    mid = (values[1:] + values[:-1]) / 2
    lo = torch.searchsorted(mid, x.contiguous())                 # mids below x: x on a mid goes down
    on = (lo < len(mid)) & (x == mid[lo.clamp(max=len(mid) - 1)])
    return torch.where(on & (lo % 2 == 1), lo + 1, lo)


def pack_fp4(x, factor):
    """Rows x [T,Hkv,D] (CPU) as pool rows [T,bytes] without their padding."""
    T, Hkv, D = x.shape
    g = x.double().view(T, Hkv, D // 16, 16)
    f32 = lambda v: torch.tensor(v, dtype=torch.float32).double()
    top = g.abs().amax(-1)
    # The definition's quotients are fp32 ones.
    step = nearest_even((top.float() / f32(6 * factor).float()).double(), e4m3_values())
    step = torch.where(top.isnan(), 127, step)
    d = (torch.cat([e4m3_values(), torch.tensor([float("nan")]).double()])[step].float() * f32(factor).float())[..., None]
    q = torch.where(d > 0, g.float() / d, torch.zeros(())).double().nan_to_num(nan=0.0)
    code = nearest_even(q.abs(), torch.tensor(LEVELS, dtype=torch.float64)) | (torch.signbit(q).long() << 3)
    code = code.view(T, Hkv * D // 2, 2)
    return torch.cat([code[..., 0] | code[..., 1] << 4, step.view(T, -1)], 1).to(torch.uint8)


def unpack_fp4(rows, Hkv, D, factor):
    """The values [...,Hkv,D] of pool rows (CPU), in 64 bits (their products fp32's, as the factor is)."""
    level = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=torch.float64)
    step = torch.cat([e4m3_values(), torch.tensor([float("nan")]).double()])
    step = torch.cat([step, -step])
    n = Hkv * D // 2
    code = rows[..., :n].long()
    code = torch.stack([code & 15, code >> 4], -1).view(*rows.shape[:-1], Hkv, D // 16, 16)
    s = step[rows[..., n:n + Hkv * D // 16].long()].view(*rows.shape[:-1], Hkv, D // 16, 1)
    return (level[code] * s * factor).view(*rows.shape[:-1], Hkv, D)


# ---------------------------------------------------------------- eviction

def select(weights, S, sinks, recent, budget):
    """Kept positions of one stream: weights [Hkv,>=S] fp32 (CPU), summed in order."""
    if S <= budget:
        return list(range(S))
    total = weights[0, :S].clone()
    for h in range(1, weights.shape[0]):
        total += weights[h, :S]
    total = total.tolist()
    key = [(-float("inf") if x != x else -x, t) for t, x in enumerate(total)]
    nan_first = [(0 if total[t] != total[t] else 1, *key[t]) for t in range(sinks, S - recent)]
    chosen = [k[2] for k in sorted(nan_first)[:budget - sinks - recent]]
    return sorted(list(range(sinks)) + chosen + list(range(S - recent, S)))
