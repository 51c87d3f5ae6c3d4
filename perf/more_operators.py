"""Operators that keep a long cache small, as cases that can be timed and compared.

Six kinds of case, each a call that a serving loop makes over grouped key heads:

  window   gqa_verify_attn_window / _paged: tree-masked attention over the first tokens and a sliding window
  append4  gqa_cache_append_fp4: new rows into a pool held in 4 bits, and the values that it then holds
  attend4  gqa_verify_attn_fp4_paged: tree-masked attention over such a pool
  weights  gqa_attn_weights_paged: the attention weight that each cached key got, added up
  select   evict_select: which keys of each stream stay, by that weight
  compact  gqa_cache_compact: the rows that stay move together

With ``own`` false, ``run`` computes them with elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

BF16, FP16 = "bf16", "fp16"
DEV = "cuda"


def listed():
    return [
        # One long stream, 9 drafts, the last 1,024 tokens and 4 first ones: the latency of a short call.
        dict(name="window_q9_w1024", kind="window", B=1, q=9, H=64, Hkv=8, D=128, lo=65536, hi=65536, window=1024, sinks=4,
             page=0, type=BF16),
        # Plain decoding of a ragged batch on 16-row pages; many streams are longer than the window.
        dict(name="window_decode64", kind="window", B=64, q=1, H=64, Hkv=8, D=128, lo=1024, hi=32768, window=4096, sinks=4,
             page=16, type=BF16),
        # The framework's ragged batch with the narrow heads of a small drafter, a whole page of first tokens.
        dict(name="window_ragged8_d64", kind="window", B=8, q=9, H=32, Hkv=8, D=64, lo=1024, hi=32768, window=8192, sinks=64,
             page=64, type=FP16),
        # The drafts' rows of 8 streams go into a 4-bit pool.
        dict(name="append4_t72", kind="append4", T=72, rows=65600, Hkv=8, D=128, type=BF16, pad=0),
        # A prompt chunk's keys and values, cut out of a fused projection, with padding tokens behind it.
        dict(name="append4_t32768", kind="append4", T=32768, rows=131072, Hkv=8, D=128, type=BF16, pad=517),
        # The framework's long-context workload over a 4-bit cache: one stream, 9 drafts, 64k keys.
        dict(name="attend4_q9_p65536", kind="attend4", B=1, q=9, H=64, Hkv=8, D=128, lo=65536, hi=65536, page=64, type=BF16),
        # Plain decoding of a ragged batch over a 4-bit cache, 16-row pages.
        dict(name="attend4_decode64", kind="attend4", B=64, q=1, H=64, Hkv=8, D=128, lo=1024, hi=32768, page=16, type=BF16),
        # What the keys of one long stream got from 9 drafts.
        dict(name="weights_q9_p65536", kind="weights", B=1, q=9, H=64, Hkv=8, D=128, lo=65536, hi=65536, page=64, type=BF16),
        # The same for a decoding batch.
        dict(name="weights_decode64", kind="weights", B=64, q=1, H=64, Hkv=8, D=128, lo=1024, hi=32768, page=16, type=FP16),
        # One long stream is cut to a quarter.
        dict(name="select_b1_s65536", kind="select", B=1, Hkv=8, lo=65536, hi=65536, budget=16384, sinks=4, recent=1024),
        # A batch around its budget: some streams are within it.
        dict(name="select_b64_ragged", kind="select", B=64, Hkv=8, lo=1024, hi=32768, budget=4096, sinks=4, recent=512),
        # The rows that stay of 8 streams, keys and values.
        dict(name="compact_b8_s32768", kind="compact", B=8, Hkv=8, D=128, lo=16384, hi=32768, budget=8192, sinks=4, recent=1024,
             page=64, type=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["window", "window", "append4", "attend4", "attend4", "weights", "select", "compact"])
    if kind in ("window", "attend4", "weights"):
        while True:
            Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
            lo = _log(rng, 1, 32768)
            c = dict(kind=kind, B=_log(rng, 1, 64), q=_log(rng, 1, 64), H=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
                     lo=lo, hi=max(lo, _log(rng, 1, 65536)), page=rng.choice([1, 16, 24, 64, 100, 256]),
                     type=rng.choice([BF16, FP16]))
            if kind == "window":
                c["window"], c["sinks"] = _log(rng, 1, 16384), rng.choice([0, 1, 4, 64, _log(rng, 1, 1000)])
                c["page"] = rng.choice([0, c["page"]])
            w = work(c)
            if c["B"] * c["H"] * c["q"] * (c["hi"] + c["q"]) <= 1.3e8 and w["bytes"] <= 6e8 and w["flops"] <= 1.9e10:
                return c
    if kind == "append4":
        T, Hkv = _log(rng, 1, 32768), rng.choice([1, 2, 3, 8])
        return dict(kind=kind, T=T, rows=T + _log(rng, 1, 65536), Hkv=Hkv, D=rng.choice([64, 128]),
                    type=rng.choice([BF16, FP16]), pad=rng.randrange(0, T))
    lo = _log(rng, 1, 32768)
    c = dict(kind=kind, B=_log(rng, 1, 64 if kind == "select" else 8), Hkv=rng.choice([1, 2, 8]), lo=lo,
             hi=_log(rng, lo, 32768), budget=_log(rng, 1, 16384))
    c["sinks"] = rng.choice([0, min(4, c["budget"])])
    c["recent"] = rng.randrange(0, c["budget"] - c["sinks"] + 1)
    if kind == "compact":
        c.update(D=rng.choice([64, 128]), page=rng.choice([1, 16, 24, 64]), type=rng.choice([BF16, FP16]))
    return c


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], even over the logarithm: the case alone fixes them."""
    return np.array([int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)], dtype=np.int64)


def _head_bytes(D):
    """Bytes that the D values of a head take in 4 bits: the codes, and a scale for every 16."""
    return D // 2 + D // 16


def work(case):
    c = case
    kind = c["kind"]
    if kind in ("window", "attend4", "weights"):
        lens = _spread(c["B"], c["lo"], c["hi"]) + c["q"]
        rows = c["B"] * c["q"] * c["H"]
        keys = int(lens.sum())
        if kind == "window":
            first = np.maximum(lens - c["q"] + 1 - c["window"], 0)      # of the window of a stream's first draft
            keys = int((lens - first + np.minimum(first, c["sinks"])).sum())
        flops = 4 * c["q"] * c["H"] * c["D"] * keys
        if kind == "weights":
            return {"bytes": keys * c["Hkv"] * (c["D"] * 2 + 8) + rows * (c["D"] * 2 + 4), "flops": flops // 2}
        row = 2 * _head_bytes(c["D"]) if kind == "attend4" else 4 * c["D"]
        return {"bytes": keys * c["Hkv"] * row + rows * (c["D"] * 4 + 4), "flops": flops}
    if kind == "append4":
        n = (c["T"] - c["pad"]) * 2 * c["Hkv"]
        return {"bytes": n * (4 * c["D"] + _head_bytes(c["D"])) + 4 * c["T"], "flops": 4 * n * c["D"]}
    lens = _spread(c["B"], c["lo"], c["hi"])
    keep = np.minimum(lens, c["budget"])
    if kind == "select":
        over = lens[lens > c["budget"]]
        return {"bytes": int(over.sum()) * c["Hkv"] * 4 + int(keep.sum()) * 4 + 8 * c["B"], "flops": int(over.sum()) * c["Hkv"]}
    moved = int(np.where(lens > c["budget"], keep - c["sinks"], 0).sum())
    return {"bytes": moved * (c["Hkv"] * (8 * c["D"] + 8) + 4) + 16 * c["B"], "flops": 0}


def _type(c):
    return torch.bfloat16 if c["type"] == BF16 else torch.float16


def _trees(rng, B, q):
    """Ancestor sets of random trees (parents before children) as 64-bit masks: a draft sees its ancestors and itself."""
    bits = np.zeros((B, q), dtype=np.uint64)
    for i in range(q):
        p = rng.integers(0, max(i, 1), size=B)
        bits[:, i] = (bits[np.arange(B), p] if i else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
    return bits


def _table(rng, lens, page, spare):
    """A block table for these lengths over a pool with `spare` free pages, pages in random order: (table, pages)."""
    n = -(-lens // page)
    pages = int(n.sum()) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.zeros((len(lens), int(n.max())), dtype=np.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    return table, pages


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _row_bytes(Hkv, D):
    return -(-Hkv * _head_bytes(D) // 16) * 16


def _step_up(a):
    """Magnitudes in steps of a scale to the 4-bit type's: 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())


def _quantise(x, held_scale):
    """Rows x [T,Hkv,D] as pool rows: codes (two a byte, the lower dimension in the lower half), then the scales of
    every 16 values, then zeros up to a multiple of 16 bytes.  Chunks bound the memory."""
    T, Hkv, D = x.shape
    out = torch.zeros((T, _row_bytes(Hkv, D)), dtype=torch.uint8, device=DEV)
    for t in range(0, T, 32768):
        g = x[t:t + 32768].float().view(-1, Hkv, D // 16, 16)
        n = g.shape[0]
        step = (g.abs().amax(-1) / (6.0 * held_scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
        whole = (step.float() * held_scale)[..., None]
        steps = torch.where(whole > 0, g / whole, torch.zeros_like(g))
        code = (_step_up(steps.abs()) | (torch.signbit(steps).byte() << 3)).view(n, Hkv, D // 2, 2)
        out[t:t + n, :Hkv * D // 2] = (code[..., 0] | (code[..., 1] << 4)).view(n, -1)
        out[t:t + n, Hkv * D // 2:Hkv * _head_bytes(D)] = step.view(torch.uint8).view(n, -1)
    return out


def _values(rows, Hkv, D, held_scale, dtype=torch.float32):
    """The values [...,Hkv,D] that pool rows [...,bytes] stand for."""
    lead = rows.shape[:-1]
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         dtype=dtype, device=DEV)
    code = rows[..., :Hkv * D // 2]
    code = torch.stack([code & 15, code >> 4], -1)
    step = rows[..., Hkv * D // 2:Hkv * _head_bytes(D)].contiguous().view(torch.float8_e4m3fn).to(dtype) * held_scale
    return (level[code.int()].view(*lead, Hkv, D // 16, 16) * step.view(*lead, Hkv, D // 16, 1)).view(*lead, Hkv, D)


def _evicted(c, lens, rng):
    """Kept positions of each stream of a compact case: the first, the last and random ones between, -1 behind."""
    kept = np.full((c["B"], c["budget"]), -1, dtype=np.int32)
    keep = np.minimum(lens, c["budget"])
    for b, (S, n) in enumerate(zip(lens, keep)):
        if S <= n:
            kept[b, :n] = np.arange(n)
            continue
        between = np.sort(rng.permutation(S - c["sinks"] - c["recent"])[:n - c["sinks"] - c["recent"]]) + c["sinks"]
        kept[b, :n] = np.concatenate([np.arange(c["sinks"]), between, np.arange(S - c["recent"], S)])
    return kept, keep


def prepare(case, seed):
    c = dict(case)
    kind = c["kind"]
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c}

    def normal(*shape):
        return torch.empty(shape, dtype=_type(c), device=DEV).normal_(generator=gen)

    def attention_mass(B, n):
        """Weights as attention leaves them: a few keys get most, many nothing that 32 bits still hold."""
        x = torch.empty((B, c["Hkv"], n), device=DEV).normal_(generator=gen).mul_(4).exp_()
        return torch.where(x < 0.1, torch.zeros_like(x), x)

    if kind in ("window", "attend4", "weights"):
        B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
        lens = rng.permutation(_spread(B, c["lo"], c["hi"])) + q
        bits = _trees(rng, B, q)
        s["mask"] = _gpu(np.ascontiguousarray(bits).view(np.int32).reshape(B, q, 2)[:, :, :-(-q // 32)])
        s["lens"] = _gpu(lens.astype(np.int32))
        s["q"] = normal(B, q, H, D)
        if c["page"]:
            table, pages = _table(rng, lens, c["page"], 3)
            s["table"] = _gpu(table)
            shape = (pages * c["page"], Hkv, D)
        else:
            shape = (B, int(lens.max()), Hkv, D)
        s["k"] = normal(*shape)
        s["scale"] = 1.0 / math.sqrt(D)
        if kind == "weights":
            s["lse"] = _attend(dict(s, v=s["k"]))["lse"]
            s["weights"] = attention_mass(B, s["table"].shape[1] * c["page"])
        else:
            s["v"] = normal(*shape)
            s["out"] = torch.empty((B, q, H, D), dtype=_type(c), device=DEV)
            s["lse"] = torch.empty((B, q, H), dtype=torch.float32, device=DEV)
        if kind == "attend4":
            s["k_scale"], s["v_scale"] = 0.125, 0.0625
            s["k"], s["v"] = _quantise(s["k"], s["k_scale"]), _quantise(s["v"], s["v_scale"])
    elif kind == "append4":
        T, Hkv, D = c["T"], c["Hkv"], c["D"]
        slots = rng.permutation(c["rows"])[:T].astype(np.int32)
        slots[T - c["pad"]:] = -1
        s["slots"] = _gpu(slots)
        # Keys and values as a user has them: column ranges of one projection's rows.
        fused = normal(T, 4 * Hkv, D)
        s["a"], s["b"] = fused[:, 2 * Hkv:3 * Hkv], fused[:, 3 * Hkv:]
        s["k_scale"], s["v_scale"] = 0.125, 0.0625
        s["pools"] = [torch.randint(0, 127, (c["rows"], _row_bytes(Hkv, D)), dtype=torch.uint8, device=DEV, generator=gen)
                      for _ in range(2)]
        s["held"] = [torch.zeros((T, Hkv, D), dtype=_type(c), device=DEV) for _ in range(2)]
    else:
        lens = rng.permutation(_spread(c["B"], c["lo"], c["hi"]))
        s["lens"] = _gpu(lens.astype(np.int32))
        if kind == "select":
            s["weights"] = attention_mass(c["B"], int(lens.max()))
            s["kept"] = torch.empty((c["B"], c["budget"]), dtype=torch.int32, device=DEV)
            s["keep"] = torch.empty(c["B"], dtype=torch.int32, device=DEV)
        else:
            table, pages = _table(rng, lens, c["page"], 3)
            kept, keep = _evicted(c, lens, rng)
            s["table"], s["kept"], s["keep"] = _gpu(table), _gpu(kept), _gpu(keep.astype(np.int32))
            s["pools"] = [normal(pages * c["page"], c["Hkv"], c["D"]) for _ in range(2)]
            s["weights"] = attention_mass(c["B"], table.shape[1] * c["page"])
    return s


# ---------------------------------------------------------------- plain forms

def _rows(table, page, at):
    """Pool rows of the positions `at` [B, n] of each stream."""
    return torch.gather(table.long(), 1, at // page) * page + at % page


def _seen(s, n):
    """Which of n keys each draft sees, [B,q,n]."""
    c = s["case"]
    B, q = c["B"], c["q"]
    at = torch.arange(n, device=DEV)[None]
    rel = at - (s["lens"].long() - q)[:, None]
    draft = rel.clamp(0, q - 1)
    word = torch.gather(s["mask"].long(), 2, (draft >> 5)[:, None].expand(B, q, n))
    seen = (rel < 0)[:, None] | ((((word >> (draft & 31)[:, None]) & 1) != 0) & (rel < q)[:, None])
    if c["kind"] == "window":
        # Of what a draft sees, in the cache's order, the last `window` and what lies in the first `sinks` places.
        count = seen.int().cumsum(-1, dtype=torch.int32)
        seen &= (count > count[..., -1:] - c["window"]) | (at < c["sinks"])[:, None]
    return seen


def _scores(s, k):
    """Scaled scores [B,Hkv,q,G,n] of float keys [B,n,Hkv,D], hidden ones at -inf."""
    c = s["case"]
    B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    G, n = H // Hkv, k.shape[1]
    qf = s["q"].float().view(B, q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, q * G, D)
    score = torch.matmul(qf, k.permute(0, 2, 3, 1)) * s["scale"]
    return score.view(B, Hkv, q, G, n).masked_fill(~_seen(s, n)[:, None, :, None], -math.inf)


def _cache(s, pool, held_scale):
    """A pool's rows in each stream's order, as floats [B,n,Hkv,D]."""
    c = s["case"]
    if c["page"]:
        n = s["table"].shape[1] * c["page"]
        pool = pool[_rows(s["table"], c["page"], torch.arange(n, device=DEV).expand(c["B"], n))]
    if pool.dtype is torch.uint8:
        return _values(pool, c["Hkv"], c["D"], held_scale)
    return pool.float()


def _attend(s):
    c = s["case"]
    B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    G = H // Hkv
    score = _scores(s, _cache(s, s["k"], s.get("k_scale")))
    score = score.view(B, Hkv, q * G, score.shape[-1])
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    del score
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].view(B, Hkv, q, G).permute(0, 2, 1, 3).reshape(B, q, H)
    if c["kind"] == "weights":
        return {"lse": lse}
    v = _cache(s, s["v"], s.get("v_scale")).permute(0, 2, 1, 3)
    out = (torch.matmul(p, v) / total).view(B, Hkv, q, G, D).permute(0, 2, 1, 3, 4).reshape(B, q, H, D).to(s["q"].dtype)
    return {"out": out, "lse": lse}


def _weights(s):
    c = s["case"]
    B, q, H, Hkv = c["B"], c["q"], c["H"], c["Hkv"]
    score = _scores(s, _cache(s, s["k"], None))
    lse = s["lse"].view(B, q, Hkv, H // Hkv).permute(0, 2, 1, 3)[..., None]
    s["weights"] += (score - lse).exp().sum((2, 3))
    return s["weights"]


def _append4(s):
    c = s["case"]
    n = c["T"] - c["pad"]                       # the padding tokens' slots are -1
    at = s["slots"][:n].long()
    for pool, x, held, held_scale in zip(s["pools"], (s["a"], s["b"]), s["held"], (s["k_scale"], s["v_scale"])):
        rows = _quantise(x[:n], held_scale)
        used = c["Hkv"] * _head_bytes(c["D"])
        pool[at, :used] = rows[:, :used]
        held[:n] = _values(rows, c["Hkv"], c["D"], held_scale).to(held.dtype)
    return {"k_pool": s["pools"][0], "v_pool": s["pools"][1], "k_held": s["held"][0], "v_held": s["held"][1]}


def _select(s):
    c = s["case"]
    lens = s["lens"].long()[:, None]
    n = s["weights"].shape[-1]
    total = s["weights"][:, 0].clone()
    for h in range(1, c["Hkv"]):                # one key head after the other
        total += s["weights"][:, h]
    at = torch.arange(n, device=DEV)[None]
    total = total.masked_fill((at < c["sinks"]) | (at >= lens - c["recent"]), math.inf).masked_fill(at >= lens, -1.0)
    order = total.sort(dim=-1, descending=True, stable=True).indices[:, :c["budget"]]
    m = order.shape[1]
    j = torch.arange(m, device=DEV)[None]
    keep = lens.clamp(max=c["budget"])
    order = torch.where(j < keep, order, n).sort(dim=-1).values
    s["kept"].fill_(-1)
    s["kept"][:, :m] = torch.where(j < keep, order, -1).int()
    s["keep"].copy_(keep[:, 0])
    return {"kept": s["kept"], "keep_lens": s["keep"]}


def _compact(s):
    c = s["case"]
    n = s["weights"].shape[-1]
    keep = s["keep"].long()[:, None]
    j = torch.arange(c["budget"], device=DEV).expand(c["B"], c["budget"])[:, :n]
    to_move = j < keep
    src = torch.where(to_move, s["kept"][:, :n].long(), torch.zeros_like(j))
    dst = torch.where(to_move, j, torch.zeros_like(j))
    b, i = to_move.nonzero(as_tuple=True)
    src_rows, dst_rows = _rows(s["table"], c["page"], src)[b, i], _rows(s["table"], c["page"], dst)[b, i]
    for p in s["pools"]:
        p[dst_rows] = p[src_rows]
    moved = torch.gather(s["weights"], 2, src[:, None].expand(-1, c["Hkv"], -1))
    at = torch.arange(n, device=DEV)[None]
    behind = ((at >= keep) & (at < s["lens"].long()[:, None]))[:, None]
    s["weights"][:, :, :j.shape[1]] = torch.where(to_move[:, None], moved, s["weights"][:, :, :j.shape[1]])
    s["weights"].masked_fill_(behind, 0.0)
    return {"k_pool": s["pools"][0], "v_pool": s["pools"][1], "weights": s["weights"]}


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import mla_verify_attention_gb300 as mva
    c = s["case"]
    kind = c["kind"]
    if kind in ("window", "attend4"):
        if "workspace" not in s:
            size = mva.gqa_workspace_size if kind == "window" else mva.gqa_fp4_workspace_size
            s["workspace"] = torch.empty(size(c["B"], c["q"], c["H"], c["Hkv"], c["D"]), dtype=torch.uint8, device=DEV)
        into = dict(out=s["out"], lse=s["lse"], workspace=s["workspace"])
        if kind == "attend4":
            out, lse = mva.gqa_verify_attn_fp4_paged(s["q"], s["k"], s["v"], c["Hkv"], s["table"], c["page"], s["lens"],
                                                     s["mask"], s["scale"], s["k_scale"], s["v_scale"], **into)
        elif c["page"]:
            out, lse = mva.gqa_verify_attn_window_paged(s["q"], s["k"], s["v"], s["table"], c["page"], s["lens"], s["mask"],
                                                        s["scale"], c["window"], c["sinks"], **into)
        else:
            out, lse = mva.gqa_verify_attn_window(s["q"], s["k"], s["v"], s["lens"], s["mask"], s["scale"], c["window"],
                                                  c["sinks"], **into)
        return {"out": out, "lse": lse}
    if kind == "weights":
        mva.gqa_attn_weights_paged(s["q"], s["k"], s["table"], c["page"], s["lens"], s["mask"], s["lse"], s["scale"],
                                   s["weights"])
        return s["weights"]
    if kind == "append4":
        mva.gqa_cache_append_fp4(s["pools"][0], s["pools"][1], s["a"], s["b"], s["slots"], s["k_scale"], s["v_scale"],
                                 k_held=s["held"][0], v_held=s["held"][1])
        return {"k_pool": s["pools"][0], "v_pool": s["pools"][1], "k_held": s["held"][0], "v_held": s["held"][1]}
    if kind == "select":
        if "workspace" not in s:
            n = mva.evict_workspace_size(c["B"], s["weights"].shape[2])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        mva.evict_select(s["weights"], s["lens"], c["sinks"], c["recent"], s["kept"], s["keep"], workspace=s["workspace"])
        return {"kept": s["kept"], "keep_lens": s["keep"]}
    mva.gqa_cache_compact(s["pools"][0], s["pools"][1], s["table"], c["page"], s["lens"], s["kept"], s["keep"],
                          weights=s["weights"])
    return {"k_pool": s["pools"][0], "v_pool": s["pools"][1], "weights": s["weights"]}


def run(state):
    # (weights adds to its sums, and compact works in place: another pass adds, or moves the same rows, once more.)
    if own:
        return _own(state)
    return {"window": _attend, "attend4": _attend, "weights": _weights, "append4": _append4, "select": _select,
            "compact": _compact}[state["case"]["kind"]](state)


# ---------------------------------------------------------------- 64 bits

def _seen_exact(c, words, b, n):
    """[q,n] truth values of stream b, draft by draft."""
    q = c["q"]
    seen = np.zeros((q, n), dtype=bool)
    for i in range(q):
        row = np.ones(n, dtype=bool)
        for j in range(q):
            row[n - q + j] = bool((int(words[b, i, j // 32]) >> (j % 32)) & 1)
        if c["kind"] == "window":
            at = np.flatnonzero(row)
            row[at[:max(len(at) - c["window"], 0)]] = False
            first = at[at < c["sinks"]]
            row[first] = True
        seen[i] = row
    return seen


def _held_exact(x, held_scale):
    """What the values x [T,Hkv,D] become in 4 bits, in 64 bits: the nearest of the type's values to x in steps."""
    g = x.double().view(*x.shape[:2], -1, 16)
    step = (g.abs().amax(-1, keepdim=True) / (6 * held_scale)).clamp(max=448)
    # The 8-bit scale: three bits behind the leading one, whole multiples of 2^-9 below 2^-6, ties to even.
    ulp = torch.exp2(torch.floor(torch.log2(step.clamp_min(2.0 ** -6))) - 3)
    step = torch.round(step / ulp) * ulp * held_scale
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    best, off = torch.zeros_like(g), g.abs()
    for i in range(1, 8):
        d = (g.abs() - level[i] * step).abs()
        closer = d < off if i % 2 else d <= off
        best, off = torch.where(closer, level[i] * step, best), torch.minimum(d, off)
    return (torch.where(g < 0, -best, best)).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    kind = c["kind"]
    if kind == "select":
        return None
    if kind == "append4":
        n = c["T"] - c["pad"]
        held = [h.double() for h in s["held"]]
        for h, x, f in zip(held, (s["a"], s["b"]), (s["k_scale"], s["v_scale"])):
            for t in range(0, n, 8192):
                h[t:min(t + 8192, n)] = _held_exact(x[t:min(t + 8192, n)], f)
        return {"k_pool": None, "v_pool": None, "k_held": held[0], "v_held": held[1]}
    if kind == "compact":
        table, kept, keep, lens = (s[x].cpu().numpy() for x in ("table", "kept", "keep", "lens"))
        pools = [p.double() for p in s["pools"]]
        weights = s["weights"].double()
        row = lambda b, t: table[b, t // c["page"]].astype(np.int64) * c["page"] + t % c["page"]
        for b, n in enumerate(keep):
            src, dst = _gpu(row(b, kept[b, :n].astype(np.int64))), _gpu(row(b, np.arange(n)))
            for p in pools:
                p.index_copy_(0, dst, p[src])
            new = weights[b][:, _gpu(kept[b, :n].astype(np.int64))]
            weights[b, :, :lens[b]] = 0
            weights[b, :, :n] = new
        return {"k_pool": pools[0], "v_pool": pools[1], "weights": weights}
    B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    G = H // Hkv
    words = s["mask"].cpu().numpy().view(np.uint32)
    table = s["table"].cpu().numpy() if c["page"] else None
    out = torch.empty((B, q, H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, q, H), dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if kind == "weights" else None
    for b, n in enumerate(s["lens"].tolist()):
        hidden = torch.from_numpy(~_seen_exact(c, words, b, n)).to(DEV).repeat_interleave(G, 0)

        def cache(pool, held_scale):
            if c["page"]:
                t = np.arange(n)
                pool = pool[_gpu(table[b, t // c["page"]].astype(np.int64) * c["page"] + t % c["page"])]
            else:
                pool = pool[b, :n]
            return _values(pool, Hkv, D, held_scale, torch.float64) if kind == "attend4" else pool

        k = cache(s["k"], s.get("k_scale"))
        v = cache(s["v"], s.get("v_scale")) if kind != "weights" else None
        for h in range(Hkv):
            x = s["q"][b, :, h * G:(h + 1) * G].double().reshape(q * G, D) @ k[:, h].double().t() * s["scale"]
            x[hidden] = -math.inf
            if kind == "weights":
                given = s["lse"][b, :, h * G:(h + 1) * G].double().reshape(q * G, 1)
                weights[b, h, :n] += torch.exp(x - given).sum(0)
                continue
            z = torch.logsumexp(x, 1)
            y = torch.exp(x - z[:, None]) @ v[:, h].double()
            out[b, :, h * G:(h + 1) * G] = y.view(q, G, D)
            lse[b, :, h * G:(h + 1) * G] = z.view(q, G)
    return weights if kind == "weights" else {"out": out, "lse": lse}
