"""What is measured of the paged compressed cache: its cases, their inputs, and the operators in plain torch.

A page holds the 64-byte blocks of `page` tokens of every KV head; a sequence is a row of page numbers and a length.
Five operators work on it: rope (rotary positions), paged_append (keys rotated, keys and values encoded into their
pages), paged_attention (a chunk of new tokens, or one, over the pages), copy_pages and compact_pages (kept tokens
moved together). `own` chooses between the plain forms below and the framework's calls.

The plain forms follow the block format's definition: decoded values are bf16 numbers by that definition, the
encoder's decisions are fp32 operations that round one by one, and everything else is fp32, rounded once at the end.
"""
import functools
import heapq
import random

import numpy as np
import torch

own = False

DIM = 128       # head dimension = values of a block
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    llama = {"heads": 8, "group": 4}  # 32 query and 8 KV heads of 128: this repository's KV-cache shape
    return [
        # one user, one token, a short prompt behind it: nothing but latency
        {"name": "attend 1 new over 650", "op": "attend", "batch": 1, "new": 1, "kv": 650, "page": 16, "window": 0, "lse": False, **llama},
        # a decode step of a small batch at different lengths: the cache's own size, [8, 8, 4096, 128]
        {"name": "attend 8x1 new over 4096", "op": "attend", "batch": 8, "new": 1, "kv": 4096, "page": 64, "window": 0, "lse": False, **llama},
        # a batch that mixes prompt pieces with single tokens: 5 query heads a KV head, pages that end inside a tile, a window, and the log-sum for a later merge
        {"name": "attend mixed odd", "op": "attend", "batch": 9, "new": 301, "kv": 2900, "page": 48, "window": 1000, "lse": True, "heads": 4, "group": 5},
        # a piece of a prompt behind a long context
        {"name": "attend 500 new over 131072", "op": "attend", "batch": 1, "new": 500, "kv": 131072, "page": 64, "window": 0, "lse": False, **llama},
        # prompt processing in large pieces: the products bound it
        {"name": "attend 4096 new over 16384", "op": "attend", "batch": 1, "new": 4096, "kv": 16384, "page": 64, "window": 0, "lse": False, **llama},
        # queries of a decode step
        {"name": "rope 8 tokens", "op": "rope", "tokens": 8, "heads": 32, "dim": 128, "rotary": 128, "interleaved": False, "inverse": False, "dtype": "bfloat16", "far": 8192},
        # queries of a long prompt, adjacent pairs, half of the head, positions far out
        {"name": "rope 8191 tokens", "op": "rope", "tokens": 8191, "heads": 32, "dim": 128, "rotary": 64, "interleaved": True, "inverse": True, "dtype": "bfloat16", "far": 131072},
        # a decode step's new token of 8 sequences
        {"name": "append 8x1", "op": "append", "batch": 8, "new": 1, "kv": 4096, "page": 64, "heads": 8, "rotary": 128, "interleaved": False},
        # prompts, ragged, half of the head rotated
        {"name": "append 4x2048", "op": "append", "batch": 4, "new": 2048, "kv": 4100, "page": 48, "heads": 8, "rotary": 64, "interleaved": True},
        # beams that fork: the last, half full page of each
        {"name": "copy 6 pages", "op": "copy", "pairs": 6, "page": 16, "heads": 8},
        # a shared prefix made private, or pages moved together
        {"name": "copy 6000 pages", "op": "copy", "pairs": 6000, "page": 64, "heads": 8},
        # tokens dropped from a long context, half of them
        {"name": "compact 3x100000", "op": "compact", "batch": 3, "kv": 100000, "page": 64, "heads": 8, "kept": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "append", "copy", "compact"])
    page, heads = rng.choice([8, 16, 24, 32, 48, 64, 100, 128]), rng.choice([1, 2, 4, 5, 8])
    if op == "attend":
        group, batch = rng.choice([1, 2, 3, 4, 5, 7, 8]), _log(rng, 1, 32)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        kv = max(new, _log(rng, 1, 131072))
        while batch > 1 and (batch * kv * heads > 1 << 20 or batch * new * kv * heads * group > 1 << 30):
            batch -= 1
        while new * kv * heads * group > 1 << 30 and heads > 1:
            heads //= 2
        while new * kv * heads * group > 1 << 30 and new > 1:
            new //= 2
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return {"op": op, "batch": batch, "new": new, "kv": kv, "page": page, "window": window, "lse": rng.random() < 0.5, "heads": heads, "group": group}
    if op == "rope":
        dim = rng.choice([64, 128, 128, 256])
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.choice([1, 5, 8, 32]), "dim": dim, "rotary": rng.choice([16, dim // 4, dim // 2, 3 * dim // 4, dim]), "interleaved": rng.random() < 0.5,
                "inverse": rng.random() < 0.3, "dtype": rng.choice(["bfloat16", "bfloat16", "float16", "float32"]), "far": _log(rng, 2048, 131072)}
    if op == "append":
        new = _log(rng, 1, 4096)
        batch = _log(rng, 1, max(1, min(32, 8192 // new)))
        return {"op": op, "batch": batch, "new": new, "kv": new + _log(rng, 1, 8192), "page": page, "heads": heads, "rotary": rng.choice([0, 32, 64, 96, 128]), "interleaved": rng.random() < 0.5}
    if op == "copy":
        return {"op": op, "pairs": _log(rng, 1, 6000), "page": rng.choice([8, 16, 24, 32, 48, 64]), "heads": heads}
    batch = rng.choice([1, 2, 3])
    return {"op": op, "batch": batch, "kv": _log(rng, 1, 100000), "page": page, "heads": heads, "kept": rng.choice([0.05, 0.5, 0.9, 1.0])}


def _lens(case):
    """(new tokens, whole length) of each sequence: the first has the case's sizes, the others lie below them."""
    rng = random.Random(1000003 * case["kv"] + 1009 * case["new"] + case["batch"])
    new, kv = [case["new"]], [case["kv"]]
    for _ in range(case["batch"] - 1):
        n = 1 if rng.random() < 0.3 else rng.randint(1, case["new"])
        new.append(n)
        kv.append(rng.randint(max(n, case["kv"] // 3), case["kv"]))
    return new, kv


# ------------------------------------------------------------------ tables of the block format
def _huffman(weights):
    """Code lengths of a prefix code; no weight under 2% of the sum, so none is longer than 8."""
    w = np.maximum(weights / weights.sum(), 0.02)
    heap = [(float(x), i, [i]) for i, x in enumerate(w)]
    lens = np.zeros(len(w), np.uint8)
    heapq.heapify(heap)
    while len(heap) > 1:
        a, b = heapq.heappop(heap), heapq.heappop(heap)
        lens[a[2] + b[2]] += 1
        heapq.heappush(heap, (a[0] + b[0], min(a[1], b[1]), a[2] + b[2]))
    assert lens.max() <= 8
    return lens


@functools.lru_cache(None)
def _tables(kind):
    """The parameters of one tensor's format, learned offline in a user's program (here: simply, from samples of the
    cache's distribution): scale, 64 patterns of 15 centroids, 4 prefix codes a pattern; and the derived tables."""
    rng = np.random.default_rng({"k": 11, "v": 12}[kind])
    scale = np.exp(rng.standard_normal((8, DIM)) * 0.5)
    scale[:, :4] *= 15.0
    x = rng.standard_normal((8, 256, DIM)) * rng.permuted(scale, axis=1)[:, None]
    x = x.reshape(-1, DIM)
    S_t = np.float32(np.abs(x).max() / 448.0)
    m = np.abs(x).argmax(1)
    u = x / x[np.arange(len(x)), m][:, None]
    rest = np.sort(np.where(np.arange(DIM)[None] == m[:, None], np.inf, u), 1)[:, :-1]
    bins = np.stack([b.mean(1) for b in np.array_split(rest, 15, axis=1)], 1)
    bins[:, 0], bins[:, 14] = rest[:, 0], rest[:, -1]
    C = bins[rng.choice(len(bins), 64, replace=False)].astype(np.float32)
    C = np.maximum.accumulate(C + np.arange(15, dtype=np.float32) * np.float32(1e-4), 1).clip(-4, 4)
    T = (C[:, :-1] + C[:, 1:]) * np.float32(0.5)
    lens = np.zeros((64, 4, 16), np.uint8)
    for p in range(64):
        h = np.bincount(np.searchsorted(T[p], rest.reshape(-1)), minlength=15).astype(np.float64)
        for b, blend in enumerate((0.0, 0.3, 0.6, 0.9)):
            lens[p, b] = _huffman(np.append((1 - blend) * h / h.sum() + blend / 15, 1 / 128))
    code, lut = np.zeros((64, 4, 16), np.int64), np.zeros((256, 256), np.int64)
    for p in range(64):
        for b in range(4):
            at, before = 0, 0
            for sym in sorted(range(16), key=lambda s: (lens[p, b, s], s)):
                n = int(lens[p, b, sym])
                at <<= n - before
                rev = int(format(at, "0%db" % n)[::-1], 2)  # the first code bit is the first of the stream
                code[p, b, sym] = rev
                lut[b * 64 + p, rev:: 1 << n] = sym | n << 4
                at, before = at + 1, n
    head = np.array([0x31434345, 1], "<u4").tobytes() + np.array([S_t], "<f4").tobytes() + bytes(4)
    blob = head + C.astype("<f4").tobytes() + lens.tobytes()
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(DEV, d)  # noqa: E731
    return {"blob": blob, "S_t": float(S_t), "C": t(C, torch.float32), "T": t(T, torch.float32), "lens": t(lens, torch.int64), "code": t(code, torch.int64), "lut": t(lut, torch.int64).reshape(-1),
            "C16": t(np.concatenate([C, np.ones((64, 1), np.float32)], 1), torch.float32).reshape(-1)}


@functools.lru_cache(None)
def _handle(kind):
    import entropy_coded_kv_b200 as ecco

    return ecco.Tables(_tables(kind)["blob"])


# ------------------------------------------------------------------ the block format, plain
def _encode(x, tab):
    """[n, 128] bf16 -> [n, 64] bytes."""
    n = x.shape[0]
    at = torch.arange(DIM, device=x.device)
    bits = x.contiguous().view(torch.int16).to(torch.int64) & 0xFFFF
    bad = (bits & 0x7F80) == 0x7F80
    x, mag = x.float().masked_fill(bad, 0.0), (bits & 0x7FFF).masked_fill(bad, 0)
    key = mag * 128 + (127 - at)
    m = 127 - key.max(1).values % 128
    is_m = at[None] == m[:, None]
    r = x.gather(1, m[:, None]).squeeze(1) / tab["S_t"]
    fp8 = r.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    s = tab["S_t"] * fp8.float()
    code, zero = fp8.view(torch.uint8).to(torch.int64), fp8.float() == 0
    u = x * (1.0 / s)[:, None]
    lo = u.masked_fill(is_m, torch.inf).min(1).values[:, None] - tab["C"][:, 0]
    hi = u.masked_fill(is_m, -torch.inf).max(1).values[:, None] - tab["C"][:, 14]
    e = lo * lo + hi * hi
    p = (e.view(torch.int32).to(torch.int64) * 64 + torch.arange(64, device=x.device)).min(1).values % 64
    sym = torch.searchsorted(tab["T"][p], u).masked_fill(is_m, 15)
    L4 = tab["lens"][p].gather(2, sym[:, None].expand(n, 4, DIM)).sum(2)
    best = (L4 * 4 + torch.arange(4, device=x.device)).min(1).values
    L, h = best // 4, best % 4
    lens, cw = tab["lens"][p, h].gather(1, sym), tab["code"][p, h].gather(1, sym)
    room = (496 - L).clamp(min=0)
    records = (room // 15).clamp(max=16)
    top = key.masked_fill(is_m, -1).topk(16, 1).values
    idx = (127 - top % 128) % 128
    q = (u.gather(1, idx) * 127.0).round().clamp(-127, 127).nan_to_num().to(torch.int64)
    slot = torch.arange(16, device=x.device)
    take = slot[None] < records[:, None]
    start = torch.cat([torch.zeros_like(m)[:, None], 16 + lens.cumsum(1) - lens, torch.where(take, 16 + L[:, None] + 15 * slot, 544)], 1).clamp(max=544)
    field = torch.cat([(code | p << 8 | h << 14)[:, None], cw, idx | (q & 0xFF) << 7], 1) << start % 32
    words = torch.zeros(n, 19, dtype=torch.int64, device=x.device)
    words.scatter_add_(1, start // 32, field & 0xFFFFFFFF).scatter_add_(1, start // 32 + 1, field >> 32)
    words = words[:, :16].masked_fill(zero[:, None], 0)
    return ((words + 2**31) % 2**32 - 2**31).to(torch.int32).view(torch.uint8)


def _words(blocks):
    return blocks.contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF


def _decode(blocks, tab):
    """[n, 64] bytes -> [n, 128] fp32 holding bf16 values. Every bit position's codeword is looked up, and the 128
    true starts follow by doubling: 1, 2, 4, ... codewords ahead."""
    w = _words(blocks)
    n = w.shape[0]
    at = torch.arange(512, device=w.device)
    two = torch.cat([w, torch.zeros_like(w[:, :1])], 1)
    pair = two[:, :-1] | (two[:, 1:] << 32)
    table = (w[:, 0] >> 8) & 255
    entry = tab["lut"][table[:, None] * 256 + ((pair.repeat_interleave(32, 1) >> at % 32) & 255)]
    nxt = at + (entry >> 4)
    jump = torch.cat([torch.where(nxt > 512, 513, nxt), torch.full_like(w[:, :2], 513)], 1)  # 512: the end, 513: clipped
    start, end = torch.full_like(w[:, :1], 16), jump
    for _ in range(7):
        start, jump = torch.cat([start, jump.gather(1, start)], 1), jump.gather(1, jump)
    last = end.gather(1, start)
    sym = entry.gather(1, start.clamp(max=511)) & 15
    code = (w[:, 0] & 255).to(torch.uint8).view(torch.float8_e4m3fn).float()
    s = torch.where(code.isnan(), 0.0, tab["S_t"] * code)
    y = (s[:, None] * tab["C16"][(table % 64)[:, None] * 16 + sym]).to(torch.bfloat16).float().masked_fill(last > 512, 0.0)
    slot = torch.arange(16, device=w.device)
    first = last[:, 127:]
    take = (first <= 512) & (slot[None] < (512 - first) // 15) & (s != 0)[:, None]
    pos = (first + 15 * slot).clamp(max=497)
    rec = (pair.gather(1, pos // 32) >> pos % 32) & 0x7FFF
    q = ((rec >> 7) ^ 0x80) - 0x80
    o = (s[:, None] * (q.float() / 127.0)).to(torch.bfloat16).float()
    y = torch.cat([y, torch.zeros_like(y[:, :1])], 1).scatter(1, torch.where(take, rec & 127, 128), o)[:, :128]
    return y.masked_fill((s == 0)[:, None], 0.0)


# ------------------------------------------------------------------ the operators, plain
def _rotate(x, table, positions, rotary, interleaved, inverse):
    """Pairs (a, b) -> (a cos - b sin, b cos + a sin) on the first `rotary` values of each head, in fp32."""
    cos, sin = table[positions.long()].unsqueeze(1).unbind(-1)
    sin = -sin if inverse else sin
    y = x.float().clone()
    r = y[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rotary // 2], r[..., rotary // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y[..., :rotary] = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return y.to(x.dtype)


def _where(st, pos):
    """Page and slot of position `pos` ([batch, n])."""
    page = st["page_table"].gather(1, (pos // st["page"]).clamp(0, st["page_table"].shape[1] - 1)).long()
    return page, pos % st["page"]


def _attend(st):
    B, H, S, n = st["batch"], st["heads"], st["kv"], st["new"]
    qlen, kvlen = st["cu_q"].long().diff(), st["kv_lens"].long()
    page, slot = _where(st, torch.arange(S, device=DEV)[None].expand(B, S).contiguous())
    k, v = (_decode(st[p + "_pages"][page, :, slot].transpose(1, 2).reshape(-1, 64), st["plain"][p]).view(B, H, S, DIM) for p in "kv")
    q = torch.zeros(B, n, H * st["group"], DIM, device=DEV)
    q[st["row_b"], st["row_i"]] = st["q"].float()
    q = q.view(B, n, H, st["group"], DIM).permute(0, 2, 3, 1, 4).reshape(B, H, -1, DIM)
    s = q @ k.transpose(-1, -2) * st["scale"]
    at, key = (kvlen - qlen)[:, None, None] + torch.arange(n, device=DEV)[:, None], torch.arange(S, device=DEV)
    hide = (key > at) | (key <= at - st["window"] if st["window"] else False)
    s = s.view(B, H, st["group"], n, S).masked_fill_(hide[:, None, None], -torch.inf)
    top = s.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, -1, S) @ v).view(B, H, st["group"], n, DIM) / total.clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, -1, DIM)[st["row_b"], st["row_i"]].to(torch.bfloat16)
    if not st["lse"]:
        return out
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, -1)[st["row_b"], st["row_i"]]
    return {"out": out, "lse": lse}


def _append(st):
    qlen, kvlen = st["cu_q"].long().diff(), st["kv_lens"].long()
    pos = (kvlen - qlen)[st["row_b"]] + st["row_i"]
    page = st["page_table"][st["row_b"], pos // st["page"]].long()
    k = _rotate(st["k"], st["table"], pos, st["rotary"], st["interleaved"], False) if st["rotary"] else st["k"]
    for name, x in (("k", k), ("v", st["v"])):
        st[name + "_pages"][page, :, pos % st["page"]] = _encode(x.reshape(-1, DIM), st["plain"][name]).view(*x.shape[:2], 64)
    return [st["k_pages"], st["v_pages"]]


def _compact(st):
    S = st["kv"]
    at = torch.arange(S, device=DEV)
    keep = st["keep"] & (at[None] < st["kv_lens"][:, None])
    page, slot = _where(st, at[None].expand(st["batch"], S).contiguous())
    to = (keep.long().cumsum(1) - 1).clamp(min=0)
    to_page, to_slot = st["dst_table"].gather(1, to // st["page"]).long()[keep], (to % st["page"])[keep]
    page, slot = page[keep], slot[keep]
    for name in "kv":
        st[name + "_pages"][to_page, :, to_slot] = st[name + "_pages"][page, :, slot]
    return [st["k_pages"], st["v_pages"], keep.sum(1, dtype=torch.int32)]


# ------------------------------------------------------------------ inputs
def _rope_table(far, rotary):
    """cos and sin of position / 10000^(2i / rotary), from fp64 angles."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, device=DEV, dtype=torch.float64) / rotary)
    a = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float()


def _cache_values(g, tokens, heads):
    """Keys or values [tokens, heads, 128]: a spread of channel scales, 4 outlier channels a head."""
    scale = torch.exp(torch.randn(heads, DIM, generator=g, device=DEV) * 0.5)
    scale.scatter_(1, torch.rand(heads, DIM, generator=g, device=DEV).topk(4, 1).indices, 15.0)
    return (torch.randn(tokens, heads, DIM, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _pool(g, pages, heads, page, kind):
    """Pages filled with encoded blocks of the cache's distribution: 4,096 tokens of each head, laid over the pages in
    another order for each head and page."""
    base = _encode(_cache_values(g, 4096, heads).reshape(-1, DIM), _tables(kind)).view(4096, heads, 64)
    pick = torch.randint(0, 4096, (pages, heads, page), generator=g, device=DEV)
    return base[pick, torch.arange(heads, device=DEV)[:, None]].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "rope":
        dtype = getattr(torch, case["dtype"])
        x = torch.randn(case["tokens"], case["heads"], case["dim"], generator=g, device=DEV).to(dtype)
        positions = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=DEV, dtype=torch.int32)
        return {**case, "x": x, "positions": positions, "table": _rope_table(case["far"], case["rotary"])}
    heads, page = case["heads"], case["page"]
    if op == "copy":
        pages = 2 * case["pairs"] + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
        src, dst = order[: case["pairs"]].contiguous(), order[case["pairs"]: 2 * case["pairs"]].contiguous()
        return {**case, "k_pages": _pool(g, pages, heads, page, "k"), "v_pages": _pool(g, pages, heads, page, "v"), "src": src, "dst": dst}
    batch, kv = case["batch"], case["kv"]
    if op == "compact":
        new, kvl = [1] * batch, [kv - 7 * b if kv > 7 * b else 1 for b in range(batch)]
    else:
        new, kvl = _lens(case)
    width = -(-kv // page)
    sets = 2 if op == "compact" else 1
    pages = sets * batch * width + 1
    order = torch.randperm(pages, generator=g, device=DEV)[: sets * batch * width].to(torch.int32).view(sets, batch, width)
    st = {**case, "k_pages": _pool(g, pages, heads, page, "k"), "v_pages": _pool(g, pages, heads, page, "v"), "page_table": order[0].contiguous(),
          "kv_lens": torch.tensor(kvl, dtype=torch.int32, device=DEV), "plain": {"k": _tables("k"), "v": _tables("v")}}
    if op == "compact":
        st["keep"] = torch.rand(batch, kv, generator=g, device=DEV) < case["kept"]
        st["dst_table"] = order[1].contiguous()
        return st
    tokens = sum(new)
    st["cu_q"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    st["row_b"] = torch.repeat_interleave(torch.arange(batch), torch.tensor(new)).to(DEV)
    st["row_i"] = torch.cat([torch.arange(n) for n in new]).to(DEV)
    if op == "attend":
        st["q"] = torch.randn(tokens, heads * case["group"], DIM, generator=g, device=DEV).to(torch.bfloat16)
        st["scale"] = DIM**-0.5
    else:
        st["k"], st["v"] = _cache_values(g, tokens, heads), _cache_values(g, tokens, heads)
        st["table"] = _rope_table(kv, case["rotary"]) if case["rotary"] else None
    if own:
        st["own"] = {"k": _handle("k"), "v": _handle("v")}
        if op == "attend":
            import entropy_coded_kv_b200 as ecco

            need = ecco.paged_attention_workspace_bytes(batch, heads, case["group"], case["new"], case["kv"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def run(st):
    if own:
        import entropy_coded_kv_b200 as ecco

        if st["op"] == "rope":
            return ecco.rope(st["x"], st["table"], st["positions"], interleaved=st["interleaved"], inverse=st["inverse"])
        if st["op"] == "copy":
            ecco.copy_pages(st["k_pages"], st["v_pages"], st["src"], st["dst"])
            return [st["k_pages"], st["v_pages"]]
        if st["op"] == "compact":
            return [st["k_pages"], st["v_pages"], ecco.compact_pages(st["k_pages"], st["v_pages"], st["page_table"], st["kv_lens"], st["keep"], st["dst_table"])]
        at = (st["k_pages"], st["v_pages"], st["own"]["k"], st["own"]["v"], st["page_table"], st["kv_lens"], st["cu_q"])
        if st["op"] == "append":
            ecco.paged_append(st["k"], st["v"], *at, rope=st["table"], interleaved=st["interleaved"])
            return [st["k_pages"], st["v_pages"]]
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV) if st["lse"] else None
        out = ecco.paged_attention(st["q"], *at, st["scale"], max_q=st["new"], max_kv=st["kv"], window=st["window"], lse=lse, workspace=st["workspace"])
        return {"out": out, "lse": lse} if st["lse"] else out
    if st["op"] == "rope":
        return _rotate(st["x"], st["table"], st["positions"], st["rotary"], st["interleaved"], st["inverse"])
    if st["op"] == "copy":
        for name in "kv":
            st[name + "_pages"][st["dst"].to(DEV).long()] = st[name + "_pages"][st["src"].to(DEV).long()]
        return [st["k_pages"], st["v_pages"]]
    return {"attend": _attend, "append": _append, "compact": _compact}[st["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(new, kv, window):
    """Pairs (new token, key) that the mask leaves, and the keys that any new token sees."""
    first = kv - new
    at = np.arange(first, kv, dtype=np.int64)
    low = np.maximum(0, at - window + 1) if window else np.zeros_like(at)
    return int((at + 1 - low).sum()), kv - int(low[0])


def work(case):
    op = case["op"]
    if op == "rope":
        size = 4 if case["dtype"] == "float32" else 2
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + case["tokens"] * (4 + 4 * case["rotary"]), "flops": 3 * n * case["rotary"]}
    if op == "copy":
        return {"bytes": 4 * case["pairs"] * case["page"] * case["heads"] * 64, "flops": 0}
    if op == "compact":
        tokens = sum(case["kv"] - 7 * b if case["kv"] > 7 * b else 1 for b in range(case["batch"]))
        return {"bytes": tokens + 4 * case["kept"] * tokens * case["heads"] * 64, "flops": 0}
    new, kv = _lens(case)
    if op == "append":
        return {"bytes": sum(new) * (2 * case["heads"] * (256 + 64) + 4 * case["rotary"]), "flops": sum(new) * case["heads"] * 3 * case["rotary"]}
    heads = case["heads"] * case["group"]
    seen = [_seen(n, s, case["window"]) for n, s in zip(new, kv)]
    bytes_ = sum(128 * case["heads"] * keys for _, keys in seen) + sum(new) * heads * (2 * 256 + 4 * case["lse"])
    return {"bytes": bytes_, "flops": sum(4 * DIM * heads * pairs for pairs, _ in seen)}


# ------------------------------------------------------------------ in 64 bits
def _walk(blocks, tab):
    """[n, 64] bytes -> [n, 128] fp64: the stream read codeword by codeword, by the code's lengths alone."""
    bits = ((blocks[:, :, None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).reshape(-1, 512).to(torch.int64)
    bits = torch.cat([bits, torch.zeros_like(bits[:, :64])], 1)
    n = bits.shape[0]
    number = lambda pos, width: sum(bits.gather(1, (pos + i)[:, None]).squeeze(1) << i for i in range(width))  # noqa: E731
    zero = torch.zeros(n, dtype=torch.int64, device=DEV)
    code, p, h = number(zero, 8), number(zero + 8, 6), number(zero + 14, 2)
    exp, frac = (code >> 3) & 15, (code & 7).double()
    fp8 = torch.where(exp > 0, (1 + frac / 8) * torch.exp2(exp.double() - 7), frac / 8 * 2.0**-6) * (1.0 - 2.0 * (code >> 7))
    s = torch.where((code & 127) == 127, 0.0, fp8) * tab["S_t"]  # exact: 24 bits by 4
    s = s.float().double()
    lens, words = tab["lens"][p, h], tab["code"][p, h]
    cents = torch.cat([tab["C"], torch.ones_like(tab["C"][:, :1])], 1).double()[p]
    y, pos, open_ = torch.zeros(n, DIM, dtype=torch.float64, device=DEV), zero + 16, torch.ones_like(zero, dtype=torch.bool)
    for i in range(DIM):
        ahead = number(pos, 8)
        sym = ((ahead[:, None] & ((1 << lens) - 1)) == words).to(torch.int64).argmax(1)
        step = lens.gather(1, sym[:, None]).squeeze(1)
        open_ = open_ & (pos + step <= 512)
        y[:, i] = torch.where(open_, s * cents.gather(1, sym[:, None]).squeeze(1), 0.0)
        pos = torch.where(open_, pos + step, pos)
    rows = torch.arange(n, device=DEV)
    for k in range(16):
        take = open_ & (pos + 15 * (k + 1) <= 512)
        at = torch.where(take, pos + 15 * k, 0)
        index, q = number(at, 7), number(at + 7, 8)
        o = (q - 256 * (q >> 7)).double() / 127.0
        y[rows[take], index[take]] = (s * o.float().double())[take]
    return y.float().to(torch.bfloat16).double()  # the definition's own rounding of a decoded value


def exact(case, seed):
    if case["op"] not in ("rope", "attend"):
        return None  # bytes only
    st = prepare(case, seed)
    if case["op"] == "rope":
        half = case["rotary"] // 2
        x = st["x"].double()
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(x[..., a], x[..., b])
        turn = torch.complex(*st["table"].double()[st["positions"].long()].unbind(-1))
        z = z * (turn.conj() if case["inverse"] else turn)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
        return x
    new, kv = _lens(case)
    if case["heads"] * sum(kv) > 1100000:
        return None
    out, lse, row = [], [], 0
    for b in range(case["batch"]):
        at = torch.arange(kv[b], device=DEV)
        pages = st["page_table"][b].long()[at // case["page"]]
        k, v = (torch.cat([_walk(part, _tables(t)) for part in st[t + "_pages"][pages, :, at % case["page"]].reshape(-1, 64).split(1 << 17)]).view(kv[b], case["heads"], DIM) for t in "kv")
        o, z = torch.zeros(new[b], case["heads"] * case["group"], DIM, dtype=torch.float64, device=DEV), torch.zeros(new[b], case["heads"] * case["group"], dtype=torch.float64, device=DEV)
        last = torch.arange(kv[b] - new[b], kv[b], device=DEV)[:, None]
        see = (at <= last) & ((at > last - case["window"]) if case["window"] else True)
        for j in range(case["heads"] * case["group"]):
            h = j // case["group"]
            for r in torch.arange(new[b], device=DEV).split(1024):
                s = torch.where(see[r], st["q"][row + r, j].double() @ k[:, h].T * st["scale"], -torch.inf)
                z[r, j] = torch.logsumexp(s, 1)
                o[r, j] = torch.softmax(s, 1) @ v[:, h]
        out.append(o)
        lse.append(z)
        row += new[b]
    return {"out": torch.cat(out), "lse": torch.cat(lse)} if case["lse"] else torch.cat(out)
