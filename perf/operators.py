"""The operators of a verify step around its attention, as cases that can be timed and compared.

Four kinds of case, each a call (or the pair of calls) that a serving loop makes:

  blocks   blocks_extend + blocks_trim: block tables and slot maps from request lengths
  append   cache_append / gqa_cache_append: new rows into a page pool by slot
  keep     cache_keep / gqa_cache_keep: the rows of an accepted draft path move together
  attend   gqa_verify_attn / gqa_verify_attn_paged: tree-masked attention of grouped query heads

With ``own`` false, ``run`` computes them with elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

BF16, FP16 = "bf16", "fp16"
LATENT, ROPE = 512, 64
DEV = "cuda"


def listed():
    return [
        # One stream, 9 drafts (8 query heads a key head), 256 keys: the latency of a short verify call.
        dict(name="attend_q9_p256", kind="attend", B=1, q=9, H=64, Hkv=8, D=128, lo=256, hi=256, page=0, type=BF16),
        # The framework's long-context workload with grouped heads: one stream, 9 drafts, 64k keys.
        dict(name="attend_q9_p65536", kind="attend", B=1, q=9, H=64, Hkv=8, D=128, lo=65536, hi=65536, page=0, type=BF16),
        # Its wide tree: 33 drafts over 16k keys (264 query rows a key head).
        dict(name="attend_q33_p16384", kind="attend", B=1, q=33, H=64, Hkv=8, D=128, lo=16384, hi=16384, page=0, type=BF16),
        # Its ragged batch on 64-row pages, with the narrow heads of a small drafter.
        dict(name="attend_ragged8_d64", kind="attend", B=8, q=9, H=32, Hkv=8, D=64, lo=1024, hi=32768, page=64, type=FP16),
        # Plain decoding of a ragged batch: one token a stream, 16-row pages.
        dict(name="attend_decode64", kind="attend", B=64, q=1, H=64, Hkv=8, D=128, lo=1024, hi=32768, page=16, type=BF16),
        # The widest tree, 16 query heads a key head (1024 query rows), odd lengths: arithmetic counts.
        dict(name="attend_q64_g16", kind="attend", B=4, q=64, H=64, Hkv=4, D=128, lo=4001, hi=8191, page=0, type=FP16),
        # A verify step's bookkeeping for 8 streams: 9 drafts each, then all dropped again.
        dict(name="blocks_b8_q9", kind="blocks", B=8, new_lo=9, new_hi=9, lo=1024, hi=32768, page=64),
        # A batch of prompts admitted at once, on small pages, and released.
        dict(name="blocks_b512_prompts", kind="blocks", B=512, new_lo=17, new_hi=2048, lo=1, hi=4096, page=16),
        # The drafts' latent rows of 8 streams.
        dict(name="append_latent_t72", kind="append", T=72, rows=65600, Hkv=0, D=0, type=BF16, pad=0),
        # The keys and values of a prompt chunk, cut out of a fused projection, with padding tokens behind it.
        dict(name="append_kv_t32768", kind="append", T=32768, rows=131072, Hkv=8, D=128, type=BF16, pad=517),
        # The accepted paths of 8 streams' trees move together in the latent cache.
        dict(name="keep_latent_b8_q9", kind="keep", B=8, q=9, lo=1024, hi=8192, page=64, Hkv=0, D=0, type=BF16),
        # The same for a large batch of wide trees and separate keys and values.
        dict(name="keep_kv_b256_q33", kind="keep", B=256, q=33, lo=200, hi=600, page=16, Hkv=8, D=128, type=FP16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "blocks", "append", "keep"])
    if kind == "attend":
        while True:
            Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
            lo = _log(rng, 1, 32768)
            c = dict(kind=kind, B=_log(rng, 1, 64), q=_log(rng, 1, 64), H=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
                     lo=lo, hi=max(lo, _log(rng, 1, 65536)), page=rng.choice([0, 0, 1, 16, 24, 64, 100, 256]),
                     type=rng.choice([BF16, FP16]))
            w = work(c)
            if c["B"] * c["H"] * c["q"] * (c["hi"] + c["q"]) <= 1.3e8 and w["bytes"] <= 2.3e9 and w["flops"] <= 4.5e10:
                return c
    if kind == "blocks":
        new, lo = _log(rng, 1, 512), _log(rng, 1, 4096)
        return dict(kind=kind, B=_log(rng, 1, 512), new_lo=_log(rng, 1, new), new_hi=new, lo=lo, hi=_log(rng, lo, 4 * lo),
                    page=rng.choice([1, 16, 24, 64, 100]))
    if kind == "append":
        T, Hkv = _log(rng, 1, 32768), rng.choice([0, 1, 2, 8])
        return dict(kind=kind, T=T, rows=T + _log(rng, 1, 65536), Hkv=Hkv, D=rng.choice([64, 128]) if Hkv else 0,
                    type=rng.choice([BF16, FP16]), pad=rng.randrange(0, T))
    Hkv, lo = rng.choice([0, 1, 2, 8]), _log(rng, 1, 600)
    return dict(kind="keep", B=_log(rng, 1, 256), q=_log(rng, 1, 33), lo=lo, hi=_log(rng, lo, 600),
                page=rng.choice([1, 16, 24, 64]), Hkv=Hkv, D=rng.choice([64, 128]) if Hkv else 0, type=rng.choice([BF16, FP16]))


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], even over the logarithm: the case alone fixes them."""
    return np.array([int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)], dtype=np.int64)


def _kept(c):
    """Accepted drafts of each stream of a keep case: 1 .. q, all equally often."""
    return 1 + np.arange(c["B"]) % c["q"]


def _grown(c):
    """Lengths and new tokens of each stream of a blocks case, paired without an order between them."""
    pair = np.random.default_rng(0).permutation(c["B"])
    return _spread(c["B"], c["lo"], c["hi"]), _spread(c["B"], c["new_lo"], c["new_hi"])[pair]


def work(case):
    c = case
    if c["kind"] == "attend":
        keys = int(_spread(c["B"], c["lo"], c["hi"]).sum()) + c["B"] * c["q"]
        rows = c["B"] * c["q"] * c["H"]
        return {"bytes": keys * c["Hkv"] * c["D"] * 4 + rows * (c["D"] * 4 + 4), "flops": 4 * c["q"] * c["H"] * c["D"] * keys}
    if c["kind"] == "blocks":
        lens, new = _grown(c)
        blocks = int((-(-(lens + new) // c["page"]) + -lens // c["page"]).sum())
        return {"bytes": 4 * (4 * c["B"] + int(new.sum()) + 4 * blocks), "flops": 2 * int(new.sum())}
    width = 2 * c["Hkv"] * c["D"] if c["Hkv"] else LATENT + ROPE
    if c["kind"] == "append":
        return {"bytes": (c["T"] - c["pad"]) * width * 4 + 4 * c["T"], "flops": 0}
    return {"bytes": int(_kept(c).sum()) * width * 4, "flops": 0}


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
    """A block table for these lengths over a pool with `spare` free pages, pages in random order: (table, pages, free pages)."""
    n = -(-lens // page)
    pages = int(n.sum()) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.zeros((len(lens), int(n.max()) if len(n) else 1), dtype=np.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    return table, pages, order[at:]


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c}

    def normal(*shape):
        return torch.empty(shape, dtype=_type(c), device=DEV).normal_(generator=gen)

    if c["kind"] == "attend":
        B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
        lens = rng.permutation(_spread(B, c["lo"], c["hi"])) + q
        bits = _trees(rng, B, q)
        words = -(-q // 32)
        s["mask"] = _gpu(np.ascontiguousarray(bits).view(np.int32).reshape(B, q, 2)[:, :, :words])
        s["lens"] = _gpu(lens.astype(np.int32))
        s["q"] = normal(B, q, H, D)
        if c["page"]:
            table, pages, _ = _table(rng, lens, c["page"], 3)
            s["table"] = _gpu(table)
            s["k"], s["v"] = (normal(pages * c["page"], Hkv, D) for _ in range(2))
        else:
            s["k"], s["v"] = (normal(B, int(lens.max()), Hkv, D) for _ in range(2))
        s["out"] = torch.empty((B, q, H, D), dtype=_type(c), device=DEV)
        s["lse"] = torch.empty((B, q, H), dtype=torch.float32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(D)
    elif c["kind"] == "blocks":
        order = rng.permutation(c["B"])
        lens, new = (x[order] for x in _grown(c))
        after = -(-(lens + new) // c["page"])
        need = int((after - -(-lens // c["page"])).sum())
        table, pages, free = _table(rng, lens, c["page"], need + 8)
        s["table"] = _gpu(np.pad(table, ((0, 0), (0, int(after.max()) + 2 - table.shape[1])), constant_values=-1))
        s["free"], s["free_count"] = _gpu(free), _gpu(np.array([len(free)], dtype=np.int32))
        s["lens"], s["new"] = _gpu(lens.astype(np.int32)), _gpu(new.astype(np.int32))
        s["keep"] = s["lens"].clone()
        s["slots"] = torch.empty(int(new.sum()), dtype=torch.int32, device=DEV)
        s["pages"], s["need"] = pages, need
    elif c["kind"] == "append":
        T, Hkv, D = c["T"], c["Hkv"], c["D"]
        slots = rng.permutation(c["rows"])[:T].astype(np.int32)
        slots[T - c["pad"]:] = -1
        s["slots"] = _gpu(slots)
        if Hkv:
            # Keys and values as a user has them: column ranges of one projection's rows.
            fused = normal(T, 4 * Hkv, D)
            s["a"], s["b"] = fused[:, 2 * Hkv:3 * Hkv], fused[:, 3 * Hkv:]
            s["pools"] = [normal(c["rows"], Hkv, D) for _ in range(2)]
        else:
            fused = normal(T, LATENT + ROPE)
            s["a"], s["b"] = fused[:, :LATENT], fused[:, LATENT:]
            s["pools"] = [normal(c["rows"], LATENT + ROPE)]
    else:
        B, q, Hkv, D = c["B"], c["q"], c["Hkv"], c["D"]
        lens = rng.permutation(_spread(B, c["lo"], c["hi"])) + q
        keep = rng.permutation(_kept(c))
        path = np.full((B, q), -1, dtype=np.int32)
        for b in range(B):
            path[b, :keep[b]] = np.sort(rng.permutation(q)[:keep[b]])
        table, pages, _ = _table(rng, lens, c["page"], 3)
        s["table"], s["lens"] = _gpu(table), _gpu(lens.astype(np.int32))
        s["path"], s["keep"] = _gpu(path), _gpu(keep.astype(np.int32))
        shape = (Hkv, D) if Hkv else (LATENT + ROPE,)
        s["pools"] = [normal(pages * c["page"], *shape) for _ in range(2 if Hkv else 1)]
    return s


# ---------------------------------------------------------------- plain forms

def _rows(table, page, at):
    """Pool rows of the positions `at` [B, n] of each stream."""
    return torch.gather(table.long(), 1, at // page) * page + at % page


def _attend(s):
    c = s["case"]
    B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    G = H // Hkv
    k, v = s["k"], s["v"]
    lens = s["lens"].long()
    if c["page"]:
        n = s["table"].shape[1] * c["page"]
        at = torch.arange(n, device=DEV).expand(B, n)
        rows = _rows(s["table"], c["page"], at)
        k, v = k[rows], v[rows]
    n = k.shape[1]
    qf = s["q"].float().view(B, q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, q * G, D)
    score = torch.matmul(qf, k.permute(0, 2, 3, 1).float()) * s["scale"]
    rel = torch.arange(n, device=DEV)[None] - (lens - q)[:, None]
    draft = rel.clamp(0, q - 1)
    word = torch.gather(s["mask"].long(), 2, (draft >> 5)[:, None].expand(B, q, n))
    seen = (rel < 0)[:, None] | ((((word >> (draft & 31)[:, None]) & 1) != 0) & (rel < q)[:, None])
    score = score.view(B, Hkv, q, G, n).masked_fill(~seen[:, None, :, None], -math.inf).view(B, Hkv, q * G, n)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).float()) / total
    lse = (top + total.log())[..., 0]
    out = out.view(B, Hkv, q, G, D).permute(0, 2, 1, 3, 4).reshape(B, q, H, D).to(s["q"].dtype)
    return {"out": out, "lse": lse.view(B, Hkv, q, G).permute(0, 2, 1, 3).reshape(B, q, H)}


def _items(count, n):
    """The stream of each of the n = sum(count) items, counted stream by stream, and its number within the stream."""
    end = torch.cumsum(count, 0)
    item = torch.arange(n, device=DEV)
    b = torch.searchsorted(end, item, right=True)
    return b, item - (end - count)[b]


def _blocks(s):
    page, table, free, fc = s["case"]["page"], s["table"], s["free"], s["free_count"]
    lens, new = s["lens"].long(), s["new"].long()
    have, after = (lens + page - 1) // page, (lens + new + page - 1) // page
    # Extend: new blocks in request order from the top of the free list.
    b, i = _items(after - have, s["need"])
    table[b, have[b] + i] = free[(fc.long() - 1 - torch.arange(s["need"], device=DEV))]
    b, i = _items(new, s["slots"].numel())
    at = lens[b] + i
    s["slots"].copy_(table[b, at // page].long() * page + at % page)
    s["lens"].add_(s["new"])
    fc.sub_(s["need"])
    # Trim back to `keep`: the released blocks go back in the same order.
    lens, keep = s["lens"].long(), s["keep"].long()
    have, after = (keep + page - 1) // page, (lens + page - 1) // page
    b, i = _items(after - have, s["need"])
    free[(fc.long() + s["need"] - 1 - torch.arange(s["need"], device=DEV))] = table[b, have[b] + i]
    s["lens"].copy_(s["keep"])
    fc.add_(s["need"])
    return {n: s[n] for n in ("slots", "table", "lens", "free", "free_count")}


def _append(s):
    n = s["case"]["T"] - s["case"]["pad"]   # the padding tokens' slots are -1
    at = s["slots"][:n].long()
    if s["case"]["Hkv"]:
        s["pools"][0][at], s["pools"][1][at] = s["a"][:n], s["b"][:n]
    else:
        s["pools"][0][at] = torch.cat([s["a"][:n], s["b"][:n]], 1)
    return s["pools"]


def _keep(s):
    c = s["case"]
    start = (s["lens"].long() - c["q"])[:, None]
    j = torch.arange(c["q"], device=DEV).expand(c["B"], c["q"])
    path = torch.where(j < s["keep"][:, None], s["path"].long(), j)
    src, dst = _rows(s["table"], c["page"], start + path), _rows(s["table"], c["page"], start + j)
    for p in s["pools"]:
        p[dst] = torch.where((j < s["keep"][:, None]).view(c["B"], c["q"], *[1] * (p.dim() - 1)), p[src], p[dst])
    return s["pools"]


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import mla_verify_attention_gb300 as mva
    c = s["case"]
    if c["kind"] == "attend":
        if "workspace" not in s:
            n = mva.gqa_workspace_size(c["B"], c["q"], c["H"], c["Hkv"], c["D"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        if c["page"]:
            out, lse = mva.gqa_verify_attn_paged(s["q"], s["k"], s["v"], s["table"], c["page"], s["lens"], s["mask"],
                                                 s["scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        else:
            out, lse = mva.gqa_verify_attn(s["q"], s["k"], s["v"], s["lens"], s["mask"], s["scale"], out=s["out"],
                                           lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if c["kind"] == "blocks":
        mva.blocks_extend(s["lens"], s["new"], s["table"], c["page"], s["free"], s["free_count"], s["pages"], s["slots"])
        mva.blocks_trim(s["lens"], s["keep"], s["table"], c["page"], s["free"], s["free_count"])
        return {n: s[n] for n in ("slots", "table", "lens", "free", "free_count")}
    if c["kind"] == "append":
        if c["Hkv"]:
            mva.gqa_cache_append(s["pools"][0], s["pools"][1], s["a"], s["b"], s["slots"])
        else:
            mva.cache_append(s["pools"][0], s["a"], s["b"], s["slots"])
        return s["pools"]
    if c["Hkv"]:
        mva.gqa_cache_keep(s["pools"][0], s["pools"][1], s["table"], c["page"], s["lens"], s["path"], s["keep"])
    else:
        mva.cache_keep(s["pools"][0], s["table"], c["page"], s["lens"], s["path"], s["keep"])
    return s["pools"]


def run(state):
    # (A keep case works in place: another pass moves the same rows once more, in either form.)
    if own:
        return _own(state)
    return {"attend": _attend, "blocks": _blocks, "append": _append, "keep": _keep}[state["case"]["kind"]](state)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "blocks":
        return None
    if c["kind"] == "append":
        pools = [p.double() for p in s["pools"]]
        slots = s["slots"].tolist()
        good = [t for t, r in enumerate(slots) if r >= 0]
        at = torch.tensor([slots[t] for t in good], device=DEV)
        if c["Hkv"]:
            pools[0].index_copy_(0, at, s["a"][good].double())
            pools[1].index_copy_(0, at, s["b"][good].double())
        else:
            pools[0][:, :LATENT].index_copy_(0, at, s["a"][good].double())
            pools[0][:, LATENT:].index_copy_(0, at, s["b"][good].double())
        return pools
    table = s["table"].cpu().numpy() if c.get("page") else None
    lens = s["lens"].tolist()
    if c["kind"] == "keep":
        pools = [p.double() for p in s["pools"]]
        path, keep = s["path"].tolist(), s["keep"].tolist()
        src, dst = [], []
        for b, n in enumerate(keep):
            for j in range(n):
                for to, i in ((src, path[b][j]), (dst, j)):
                    t = lens[b] - c["q"] + i
                    to.append(int(table[b, t // c["page"]]) * c["page"] + t % c["page"])
        for p in pools:
            p.index_copy_(0, torch.tensor(dst, device=DEV), p[torch.tensor(src, device=DEV)])
        return pools
    B, q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    G = H // Hkv
    out = torch.empty((B, q, H, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, q, H), dtype=torch.float64, device=DEV)
    words = s["mask"].cpu().numpy().view(np.uint32)
    for b, n in enumerate(lens):
        seen = np.ones((q, n), dtype=bool)
        for i in range(q):
            for j in range(q):
                seen[i, n - q + j] = bool((int(words[b, i, j // 32]) >> (j % 32)) & 1)
        hidden = torch.from_numpy(~seen).to(DEV).repeat_interleave(G, 0)
        k, v = s["k"], s["v"]
        if c["page"]:
            t = np.arange(n)
            rows = torch.from_numpy(table[b, t // c["page"]].astype(np.int64) * c["page"] + t % c["page"]).to(DEV)
            k, v = k[rows], v[rows]
        else:
            k, v = k[b, :n], v[b, :n]
        for h in range(Hkv):
            x = s["q"][b, :, h * G:(h + 1) * G].double().reshape(q * G, D) @ k[:, h].double().t() * s["scale"]
            x[hidden] = -math.inf
            z = torch.logsumexp(x, 1)
            y = torch.exp(x - z[:, None]) @ v[:, h].double()
            out[b, :, h * G:(h + 1) * G] = y.view(q, G, D)
            lse[b, :, h * G:(h + 1) * G] = z.view(q, G)
    return {"out": out, "lse": lse}
