"""Workloads of the key-value cache operators: attention of a verification
round over a paged cache, rows written to the cache and read back, and the
page operators (fork, release, reserve, commit, compact).

Every case runs either in plain torch operations (own = False) or through
the package's calls (own = True) on the same buffers: the cache's pages as
the package lays them out, its page tables and its lists of free pages.

Layout of one block (32 positions of one head): keys [dim/8][32][8], then
values [4][dim][8] (8 positions innermost); int8 caches add 32 fp32 scales
of the keys and 32 of the values.  A page holds its heads' blocks,
[heads][page/32]; the pool is [layers][n_pages] pages.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f16": 1, "bf16": 30, "i8": 24}


# ------------------------------------------------------------------ cases
def listed():
    a = dict(op="attention", page=64, rot=128, rope=2, window=0, sinks=0, tree=False, ragged=False, layers=1)
    w = dict(op="attention", page=64, rot=128, rope=2, tree=False, ragged=False, layers=1)
    return [
        # a plain decode step early in a conversation: one row, one short sequence, 2560 = 20 x 128; latency counts
        dict(a, name="attn_one_short", type="f16", B=1, M=1, heads=4, group=5, dim=128, len=300),
        # the verification round itself: the current token and four drafts, 5120 = 40 x 128
        dict(a, name="attn_verify", type="f16", B=1, M=5, heads=8, group=5, dim=128, len=4099),
        # the same round at the end of a long document
        dict(a, name="attn_verify_long", type="bf16", B=1, M=5, heads=8, group=5, dim=128, len=131001),
        # a batch of sequences of different lengths and draft counts, int8 cache, large pages
        dict(a, name="attn_batch_i8", type="i8", B=16, M=5, heads=8, group=5, dim=128, len=16384, ragged=True,
             page=128),
        # draft trees of up to 16 rows, 64 query rows per key head; adjacent-pair rotation of half of a head
        dict(a, name="attn_tree", type="f16", B=4, M=16, heads=8, group=4, dim=64, len=8191, ragged=True, tree=True,
             rot=32, rope=1),
        # streaming decode: one row each, a window of 1024 and four first positions that stay
        dict(w, name="window_one", type="bf16", B=8, M=1, heads=8, group=1, dim=96, len=30000, window=1024, sinks=4,
             page=32, rot=96),
        # verification over a wide window, many sequences
        dict(w, name="window_verify", type="f16", B=32, M=5, heads=8, group=5, dim=128, len=32768, window=4096,
             sinks=64, ragged=True),
        # rows of one verification round into one layer of the cache, and read back
        dict(op="append", name="append_verify", type="i8", B=1, M=5, heads=8, dim=128, len=1000, page=64, rot=128,
             rope=2, ragged=False, layers=1),
        # prompts of a small batch into one layer
        dict(op="append", name="append_prompt", type="f16", B=4, M=3000, heads=8, dim=128, len=77, page=64, rot=128,
             rope=2, ragged=True, layers=1),
        # several candidates forked off one prompt, with their part-filled last pages, over all layers
        dict(op="fork", name="fork", type="bf16", B=15, heads=8, dim=128, len=8000, page=128, layers=36),
        # a tree round's pages: candidates forked, room reserved for the rows, accepted paths kept, the rest freed
        dict(op="round", name="tree_round", type="f16", B=4, M=16, heads=8, dim=128, len=2040, page=64, layers=64),
        # pages moved together, so that the pool's upper end is free, over all layers
        dict(op="compact", name="compact", type="f16", B=8, heads=4, dim=128, len=4096, page=64, layers=36),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "window", "window", "append", "fork", "round", "compact"])
    c = dict(type=rng.choice(["f16", "bf16", "i8"]), heads=rng.choice([1, 2, 3, 4, 8, 10]),
             dim=rng.choice([32, 64, 96, 128, 128, 160, 192, 256]), page=rng.choice([32, 64, 128, 256]))
    if kind in ("attention", "window"):
        c.update(op="attention", B=_spread(rng, 1, 32), M=rng.randint(1, 16), group=rng.choice([1, 2, 3, 4, 5, 7, 8]),
                 rope=rng.choice([0, 1, 2]), tree=rng.random() < 0.4, ragged=rng.random() < 0.6, layers=1, window=0,
                 sinks=0)
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2])
        most = 1 << 21                       # positions x heads of a call
        c["len"] = _spread(rng, 1, max(2, min(131000, most // (c["B"] * c["heads"]))))
        if kind == "window":
            c["window"], c["sinks"] = _spread(rng, 1, 8192), rng.choice([0, 1, 4, 100])
        return c
    if kind == "append":
        c.update(op="append", B=_spread(rng, 1, 16), len=_spread(rng, 1, 8000), rope=rng.choice([0, 1, 2]),
                 ragged=rng.random() < 0.5, layers=1)
        c["M"] = _spread(rng, 1, 12000 // c["B"])
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2])
        return c
    c.update(op=kind, B=_spread(rng, 2, 15), type=rng.choice(["f16", "bf16"]), layers=_spread(rng, 1, 36),
             dim=rng.choice([64, 96, 128]), heads=rng.choice([1, 2, 4, 8]))
    c["len"] = _spread(rng, 40, 8000 if kind == "fork" else 4000)
    c["layers"] = max(1, min(c["layers"], (1 << 31) // (c["B"] * c["len"] * c["heads"] * c["dim"] * 4)))
    if kind == "round":
        c["M"] = rng.randint(2, 16)
    return c


# ------------------------------------------------------- sizes of a case
def _lens(c):
    """Cached positions of each sequence: the longest first, the others
    spread over the range when the case is ragged."""
    if not c.get("ragged"):
        return [c["len"]] * c["B"]
    return [c["len"] if b == 0 else int(c["len"] * ((b * 0.6180339887) % 1.0)) for b in range(c["B"])]


def _news(c):
    if not c.get("ragged"):
        return [c["M"]] * c["B"]
    return [c["M"] if b == 0 else max(1, int(c["M"] * ((b * 0.6180339887) % 1.0))) for b in range(c["B"])]


def _width(c):
    return -(-(c["len"] + c.get("M", 0)) // c["page"])


def _block_bytes(c):
    return 64 * c["dim"] + 256 if c["type"] == "i8" else 128 * c["dim"]


def _page_bytes(c):
    return c["heads"] * (c["page"] // 32) * _block_bytes(c)


def _row_bytes(c):
    """Bytes of one position of one head: its key and its value."""
    return 2 * c["dim"] + 8 if c["type"] == "i8" else 4 * c["dim"]


def _path(c, b):
    """Rows of a tree round that are kept: 0, then some of the later ones."""
    return [m for m in range(c["M"]) if m == 0 or (m * 5 + b) % 3 == 0]


def work(c):
    if c["op"] == "attention":
        seen = rows = 0
        for n, new in zip(_lens(c), _news(c)):
            held = n + new if not c["window"] else min(n + new, c["window"] + new - 1 + min(c["sinks"], n))
            seen += held
            rows += new
        kv = seen * c["heads"] * _row_bytes(c)
        qo = 2 * rows * c["heads"] * c["group"] * c["dim"] * 4
        return {"bytes": kv + qo, "flops": 4.0 * (seen / c["B"]) * rows * c["heads"] * c["group"] * c["dim"]}
    if c["op"] == "append":
        rows = sum(_news(c)) * c["heads"]
        return {"bytes": rows * (16 * c["dim"] + 2 * _row_bytes(c)), "flops": 6.0 * rows * c["dim"]}
    if c["op"] == "fork":
        used = -(-(c["len"] % c["page"]) // 32)
        return {"bytes": c["B"] * c["layers"] * 2 * c["heads"] * used * _block_bytes(c) + 8 * c["B"] * _width(c),
                "flops": 0}
    if c["op"] == "round":
        used = -(-(c["len"] % c["page"]) // 32)
        moved = sum(sum(m != i for i, m in enumerate(_path(c, b))) for b in range(c["B"]))
        return {"bytes": c["layers"] * c["heads"] * 2 * (c["B"] * used * _block_bytes(c) + moved * _row_bytes(c))
                + 8 * c["B"] * _width(c), "flops": 0}
    # compact: each half of the sequences moves once in a pass
    return {"bytes": 2 * c["layers"] * _page_bytes(c) * _compact_moves(c), "flops": 0}


def _compact_moves(c):
    half = c["B"] // 2 * _width(c)
    rest = (c["B"] - c["B"] // 2) * _width(c)
    return 2 * min(half, rest)


# --------------------------------------------------------------- inputs
def _pages_of(c, state, lens, gen, rows):
    """Random pages for `rows` sequences of the given lengths, room for
    M more rows each; the rest of the pool on the list of free pages."""
    P, W = c["page"], _width(c)
    table = torch.full((state["seqs"], W), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(state["n_pages"], device="cuda", generator=gen).to(torch.int32)
    at = 0
    for b in range(rows):
        k = -(-(lens[b] + (c.get("M", 0) if c["op"] in ("attention", "append") else 0)) // P)
        table[b, :k] = order[at:at + k]
        at += k
    refs = torch.zeros(state["n_pages"], dtype=torch.int32, device="cuda")
    refs[order[:at].long()] = 1
    free = torch.zeros(state["n_pages"], dtype=torch.int32, device="cuda")
    free[:state["n_pages"] - at] = order[at:]
    state.update(table=table, refs=refs, free_ids=free,
                 ctl=torch.tensor([state["n_pages"] - at, 0, 0, 0], dtype=torch.int32, device="cuda"),
                 len=torch.tensor(lens + [0] * (state["seqs"] - len(lens)), dtype=torch.int32, device="cuda"))


def _pool(c, n_pages, gen):
    """A pool whose every position holds a finite row."""
    if c["type"] != "i8":
        t = torch.float16 if c["type"] == "f16" else torch.bfloat16
        x = torch.empty(c["layers"], n_pages, _page_bytes(c) // 2, dtype=t, device="cuda")
        x.normal_(generator=gen)
        return x.view(torch.uint8)
    blocks = n_pages * c["heads"] * (c["page"] // 32)
    x = torch.empty(c["layers"], blocks, _block_bytes(c), dtype=torch.uint8, device="cuda")
    codes = 64 * c["dim"]
    x[..., :codes] = torch.randint(-127, 128, (c["layers"], blocks, codes), device="cuda", generator=gen,
                                   dtype=torch.int8).view(torch.uint8)
    scale = 0.014 * (0.5 + torch.rand(c["layers"], blocks, 64, device="cuda", generator=gen))
    x[..., codes:] = scale.view(torch.uint8)
    return x.view(c["layers"], n_pages, _page_bytes(c))


def _rope_table(n_pos, rot):
    """cos and sin of every position's angles, in 64 bits and then rounded."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


def _trees(c, seed):
    """A parent among the earlier rows for every row but the first; a row
    sees itself and its ancestors."""
    r = np.random.RandomState((seed * 1000003 + 17) % (1 << 31))
    masks = np.zeros((c["B"], c["M"]), np.int64)
    for b in range(c["B"]):
        for m in range(c["M"]):
            masks[b, m] = (1 << m) | (masks[b, r.randint(0, m)] if m else 0)
    return torch.from_numpy(masks.astype(np.int32)).cuda()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = c["B"]
    lens = [c["len"]] if c["op"] in ("fork", "round") else [0] * rows if c["op"] == "compact" else _lens(c)
    s = {"case": c, "handle": None}
    W, P = _width(c), c["page"]
    if c["op"] == "fork":
        s["seqs"], s["n_pages"] = rows + 1, W + rows + 5
    elif c["op"] == "round":
        s["seqs"], s["n_pages"] = rows + 1, W + 3 * rows + 5
    elif c["op"] == "compact":
        s["seqs"], s["n_pages"] = rows, rows * W + 1 + W
    else:
        s["seqs"], s["n_pages"] = rows, sum(-(-(n + c["M"]) // P) for n in lens) + 3
    s["data"] = _pool(c, s["n_pages"], gen)
    _pages_of(c, s, lens, gen, len(lens))
    ints = dict(dtype=torch.int32, device="cuda")
    if c["op"] in ("attention", "append"):
        s["n_new"] = torch.tensor(_news(c), **ints) if c["ragged"] else None
        s["rope"] = _rope_table(W * P, c["rot"]) if c["rope"] else None
        s["tree"] = _trees(c, seed) if c.get("tree") else None
    normal = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    if c["op"] == "attention":
        s["q"] = normal(c["B"], c["M"], c["heads"] * c["group"], c["dim"]) * 1.5
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "append":
        s["k"], s["v"] = (normal(c["B"], c["M"], c["heads"], c["dim"]) for _ in "kv")
        s["k_out"], s["v_out"] = (torch.zeros_like(s["k"]) for _ in "kv")
    elif c["op"] in ("fork", "round"):
        s["src"], s["dst"] = torch.zeros(rows, **ints), torch.arange(1, rows + 1, **ints)
        if c["op"] == "round":
            paths = [_path(c, b) for b in range(rows)]
            s["path"] = torch.tensor([p + [0] * (c["M"] - len(p)) for p in paths], **ints)
            s["accepted"] = torch.tensor([len(p) - 1 for p in paths], **ints)
    else:
        s["low"], s["high"] = torch.arange(0, rows // 2, **ints), torch.arange(rows // 2, rows, **ints)
        # all sequences hold their pages, the first half of them the lower ones
        order = torch.arange(rows * W, **ints).view(rows, W)
        s["table"].copy_(order)
        s["refs"].zero_()
        s["refs"][:rows * W] = 1
        left = s["n_pages"] - rows * W
        s["free_ids"][:left] = torch.arange(s["n_pages"] - 1, rows * W - 1, -1, **ints)
        s["ctl"][0] = left
    return s


# ------------------------------------------------------ the plain forms
def _rows_of(s, c):
    """Keys and values of every page-table entry of the first B sequences,
    fp32 [B, heads, W * page, dim]; entries without a page give page 0."""
    B, W, nb, D = c["B"], _width(c), c["page"] // 32, c["dim"]
    pages = s["data"][c["layers"] - 1][s["table"][:B].clamp(min=0).long().view(-1)]
    blocks = pages.view(B, W, c["heads"], nb, _block_bytes(c))
    t = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}[c["type"]]
    half = 32 * D * (1 if t == torch.int8 else 2)
    k = blocks[..., :half].contiguous().view(t).view(B, W, c["heads"], nb, D // 8, 32, 8).float()
    v = blocks[..., half:2 * half].contiguous().view(t).view(B, W, c["heads"], nb, 4, D, 8).float()
    k = k.permute(0, 1, 2, 3, 5, 4, 6).reshape(B, W, c["heads"], nb, 32, D)
    v = v.permute(0, 1, 2, 3, 4, 6, 5).reshape(B, W, c["heads"], nb, 32, D)
    if t == torch.int8:
        d = blocks[..., 2 * half:].contiguous().view(torch.float32)
        k, v = k * d[..., :32, None], v * d[..., 32:, None]
    k, v = (x.transpose(1, 2).reshape(B, c["heads"], -1, D) for x in (k, v))
    return k, v


def _new_rows(s, c):
    """Per sequence: cached length, new rows, each row's visible new rows
    [B, M, M] and its position."""
    B, M = c["B"], c["M"]
    n = s["len"][:B].long()
    new = s["n_new"].long() if s["n_new"] is not None else torch.full_like(n, M)
    m = torch.arange(M, device="cuda")
    if s["tree"] is not None:
        sees = (s["tree"].long()[:, :, None] >> m) & 1
    else:
        sees = (m[None, :] <= m[:, None]).long().expand(B, M, M)
    pos = n[:, None] + (sees * (m[None, :] < m[:, None])).sum(-1)
    return n, new, sees.bool(), pos


def _rotate(x, pos, s, c):
    """x [B, M, heads, dim] by the angles of pos [B, M]."""
    if not c["rope"]:
        return x
    h = c["rot"] // 2
    cs = s["rope"][pos]
    co, si = cs[:, :, None, :, 0], cs[:, :, None, :, 1]
    r = x[..., :c["rot"]]
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if c["rope"] == 1 else (r[..., :h], r[..., h:])
    y0, y1 = x0 * co - x1 * si, x1 * co + x0 * si
    y = torch.stack([y0, y1], -1).flatten(-2) if c["rope"] == 1 else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., c["rot"]:]], -1)


def _attention(s, c):
    B, M, H, G, D = c["B"], c["M"], c["heads"], c["group"], c["dim"]
    k, v = _rows_of(s, c)
    n, new, sees, pos = _new_rows(s, c)
    slot = torch.arange(k.shape[2], device="cuda")
    t = slot[None, :] - n[:, None]                                     # which new row a slot is
    fresh = (t >= 0) & (t < new[:, None])
    tc = t.clamp(0, M - 1)
    kpos = torch.where(fresh, torch.gather(pos, 1, tc), slot[None, :].expand(B, -1))
    vis = (t < 0)[:, None, :] | (fresh[:, None, :] & torch.gather(sees, 2, tc[:, None, :].expand(B, M, -1)))
    if c["window"]:
        vis = vis & ((pos[:, :, None] - kpos[:, None, :] < c["window"]) | (kpos < c["sinks"])[:, None, :])
    held = vis.any(1)
    v = v * held[:, None, :, None]
    q = _rotate(s["q"], pos, s, c).view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, H, M, G, -1) / math.sqrt(D)
    x = x.masked_fill(~vis[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, M * G, -1), v).view(B, H, M, G, D) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)
    live = torch.arange(M, device="cuda")[None, :] < new[:, None]
    s["out"].copy_(torch.where(live[:, :, None, None], o, s["out"]))
    return s["out"]


def _round_away(x):
    a = x.abs()
    f = a.floor()
    return torch.copysign(f + (a - f >= 0.5).float(), x)


def _append(s, c):
    """Writes the rows, then reads them back as fp32."""
    B, M, H, D, P = c["B"], c["M"], c["heads"], c["dim"], c["page"]
    m = torch.arange(M, device="cuda")
    slot = s["len"][:B].long()[:, None] + m
    k, v = _rotate(s["k"], slot, s, c), s["v"]
    live = m < (torch.full_like(slot[:, :1], M) if s["n_new"] is None else s["n_new"][:, None])
    page = torch.gather(s["table"][:B].long(), 1, (slot // P).clamp(max=_width(c) - 1))
    block = (page[..., None] * H + torch.arange(H, device="cuda")) * (P // 32) + (slot % P // 32)[..., None]
    at = (slot % 32)[..., None, None]
    base = block[..., None] * _block_bytes(c)
    d = torch.arange(D, device="cuda")
    pool = s["data"][c["layers"] - 1].view(-1)
    size = 1 if c["type"] == "i8" else 2
    k_at = base // size + (d // 8 * 32 + at) * 8 + d % 8
    v_at = base // size + 32 * D + (at // 8 * D + d) * 8 + at % 8
    t = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}[c["type"]]
    keep = live[:, :, None, None].expand(B, M, H, D)
    if t == torch.int8:
        scale_at = base[..., 0] // 4 + 16 * D + at[..., 0]
        full = torch.full((1,), 127.0, device="cuda")      # a tensor: torch would multiply by a number's reciprocal
        for_k, for_v = (x.abs().amax(-1, keepdim=True) / full for x in (k, v))
        k, v = (_round_away(x * torch.where(f > 0, 1.0 / f, 0.0)).clamp(-127, 127) for x, f in ((k, for_k), (v, for_v)))
        keep1 = keep[..., 0]
        pool.view(torch.float32)[scale_at[keep1]] = for_k[..., 0][keep1]
        pool.view(torch.float32)[scale_at[keep1] + 32] = for_v[..., 0][keep1]
    pool.view(t)[k_at[keep]] = k.to(t)[keep]
    pool.view(t)[v_at[keep]] = v.to(t)[keep]
    back_k, back_v = pool.view(t)[k_at].float(), pool.view(t)[v_at].float()
    if t == torch.int8:
        back_k = back_k * pool.view(torch.float32)[scale_at][..., None]
        back_v = back_v * pool.view(torch.float32)[scale_at + 32][..., None]
    s["k_out"].copy_(torch.where(keep, back_k, s["k_out"]))
    s["v_out"].copy_(torch.where(keep, back_v, s["v_out"]))
    return s["k_out"], s["v_out"]


def _put(x, at, value, keep):
    """x[at] = value where keep."""
    pad = torch.cat([x.view(-1), x.new_zeros(1)])
    pad.scatter_(0, torch.where(keep, at, x.numel()).view(-1), value.to(x.dtype).expand(at.shape).reshape(-1))
    x.view(-1).copy_(pad[:-1])


def _release(s, ids):
    """Drops the pages of sequences `ids`; a page that no sequence holds any
    more goes on the free list, in the order of the last entry naming it."""
    rows = s["table"][ids.long()].long()
    held = rows >= 0
    p = rows.clamp(min=0).view(-1)
    hold = held.view(-1)
    refs = s["refs"]
    refs.index_add_(0, p, -hold.to(torch.int32))
    idx = torch.arange(p.numel(), device="cuda")
    last = torch.full((refs.numel(),), -1, dtype=torch.int64, device="cuda")
    last.scatter_reduce_(0, p, torch.where(hold, idx, -1), "amax")
    push = hold & (refs[p] == 0) & (last[p] == idx)
    _put(s["free_ids"], s["ctl"][0] + push.cumsum(0) - 1, p, push)
    s["ctl"][0] += push.sum().to(torch.int32)
    s["table"][ids.long()] = -1
    s["len"][ids.long()] = 0


def _take(s, at, want):
    """Pages off the end of the free list for the wanted entries of the
    table (flat indices `at`), in their order."""
    page = s["free_ids"][(s["ctl"][0] - want.cumsum(0)).clamp(min=0).long()]
    _put(s["table"], at, page, want)
    _put(s["refs"], page.long(), torch.ones_like(page), want)
    s["ctl"][0] -= want.sum().to(torch.int32)


def _fork(s, c):
    """dst shares src's full pages and gets a copy of its part-filled one."""
    src, dst, P, W = s["src"].long(), s["dst"].long(), c["page"], s["table"].shape[1]
    n = s["len"][src].long()
    full = n // P
    e = torch.arange(W, device="cuda")
    rows = torch.where(e < full[:, None], s["table"][src], -1)
    s["refs"].index_add_(0, rows.clamp(min=0).long().view(-1), (rows >= 0).to(torch.int32).view(-1))
    s["table"][dst] = rows
    s["len"][dst] = n.to(torch.int32)
    part = n % P > 0
    last = full.clamp(max=W - 1)
    _take(s, dst * W + last, part)
    used = -(-(c["len"] % P) // 32)                       # the blocks of the page that hold positions
    if used:
        data = s["data"].view(c["layers"], -1, c["heads"], P // 32, _block_bytes(c))
        old, new = s["table"][src, last].long(), s["table"][dst, last].long()
        data[:, new, :, :used] = data[:, old, :, :used]


def _reserve(s, ids, n, c):
    P, W = c["page"], s["table"].shape[1]
    have = s["len"][ids.long()].long()
    e = torch.arange(W, device="cuda")
    want = (e >= (-(-have // P))[:, None]) & (e < (-(-(have + n) // P))[:, None]) & (s["table"][ids.long()] < 0)
    _take(s, (ids.long()[:, None] * W + e).view(-1), want.view(-1))


def _commit(s, c):
    """Moves the kept rows together, then lengthens the sequences and frees
    the pages past their ends."""
    B, M, P, W, D, H = c["B"], c["M"], c["page"], s["table"].shape[1], c["dim"], c["heads"]
    ids = s["dst"].long()
    n, kept = s["len"][ids].long(), s["accepted"].long() + 1
    i = torch.arange(M, device="cuda")
    live = (i < kept[:, None]) & (s["path"] != i)
    src, dst = n[:, None] + s["path"].long(), n[:, None] + i
    t = torch.float16 if c["type"] == "f16" else torch.bfloat16
    pool = s["data"].view(-1).view(t)
    layer = torch.arange(c["layers"], device="cuda").view(-1, 1, 1, 1, 1) * s["n_pages"]
    head, d = torch.arange(H, device="cuda").view(-1, 1), torch.arange(D, device="cuda")

    def places(slot):
        page = torch.gather(s["table"][ids].long(), 1, (slot // P).clamp(max=W - 1))[..., None, None]
        slot = slot[..., None, None]
        base = (((layer + page) * H + head) * (P // 32) + slot % P // 32) * (64 * D)
        return base + (d // 8 * 32 + slot % 32) * 8 + d % 8, base + 32 * D + (slot % 32 // 8 * D + d) * 8 + slot % 8

    (k0, v0), (k1, v1) = places(src), places(dst)
    keep = live[None, :, :, None, None].expand(k0.shape)
    k, v = pool[k0[keep]], pool[v0[keep]]
    pool[k1[keep]], pool[v1[keep]] = k, v
    s["len"][ids] = (n + kept).to(torch.int32)
    e = torch.arange(W, device="cuda")
    rows = s["table"][ids]
    drop = ((e >= (-(-(n + kept) // P))[:, None]) & (rows >= 0)).view(-1)
    p = rows.long().view(-1)
    _put(s["free_ids"], s["ctl"][0] + drop.cumsum(0) - 1, p, drop)
    _put(s["refs"], p, torch.zeros_like(p), drop)
    s["ctl"][0] += drop.sum().to(torch.int32)
    s["table"][ids] = torch.where(drop.view(B, W), -1, rows)


def _compact(s, c):
    """Held pages above the number of held pages move to the free ones below
    it, both in ascending order."""
    n, refs = s["n_pages"], s["refs"]
    live = n - s["ctl"][0].long()
    ids = torch.arange(n, device="cuda")
    old, new = ids[(ids >= live) & (refs > 0)], ids[(ids < live) & (refs == 0)]
    to = ids.clone()
    to[old] = new
    s["data"][:, new] = s["data"][:, old]
    refs[new], refs[old] = refs[old], torch.zeros_like(refs[old])
    t = s["table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].to(torch.int32), t))
    s["free_ids"].copy_(torch.where(ids < s["ctl"][0], n - 1 - ids, s["free_ids"].long()).to(torch.int32))


def _state_of(s):
    """What a page operator leaves: the tables, the counts, and the pool."""
    t = torch.bfloat16 if s["case"]["type"] == "bf16" else torch.float16
    return s["table"], s["len"], s["refs"], s["ctl"][:1], s["data"].view(t)


# --------------------------------------------------------------- the pass
def _handle(s):
    """The package's cache object over the state's buffers, and the plan of
    its attention: made at the first pass, as a program makes them once."""
    import speculative_decoding_verification_amd as sv
    c = s["case"]
    kv = sv.KvCache(TYPES[c["type"]], c["layers"], c["heads"], c["dim"], c["page"], s["n_pages"], s["seqs"],
                    _width(c), buffers={k: s[k] for k in ("data", "table", "len", "refs", "free_ids", "ctl")})
    rope = sv.Rope(c["rope"], c["rot"], s["rope"]) if c.get("rope") else None
    plan = None
    if c["op"] == "attention":
        plan = kv.attention(c["heads"] * c["group"], c["B"], c["M"], window=c["window"], sinks=c["sinks"])
    s["handle"] = kv, plan, rope
    return s["handle"]


def run(s):
    c = s["case"]
    if own:
        kv, plan, rope = s["handle"] or _handle(s)
        if c["op"] == "attention":
            plan.run(c["layers"] - 1, s["q"], s["out"], n_new=s["n_new"], tree=s["tree"], rope=rope)
            return s["out"]
        if c["op"] == "append":
            kv.append(c["layers"] - 1, s["k"], s["v"], n_new=s["n_new"], rope=rope)
            kv.read(c["layers"] - 1, s["k_out"], s["v_out"], n_new=s["n_new"])
            return s["k_out"], s["v_out"]
        if c["op"] in ("fork", "round"):
            kv.release(s["dst"])
            kv.fork(s["src"], s["dst"])
            if c["op"] == "round":
                kv.reserve(c["M"], seq=s["dst"])
                kv.commit(c["M"], s["accepted"], seq=s["dst"], path=s["path"])
            return _state_of(s)
        kv.release(s["low"])
        kv.compact()
        kv.reserve(c["len"], seq=s["low"])
        kv.release(s["high"])
        kv.compact()
        kv.reserve(c["len"], seq=s["high"])
        return _state_of(s)
    if c["op"] == "attention":
        return _attention(s, c)
    if c["op"] == "append":
        return _append(s, c)
    if c["op"] in ("fork", "round"):
        _release(s, s["dst"])
        _fork(s, c)
        if c["op"] == "round":
            _reserve(s, s["dst"], c["M"], c)
            _commit(s, c)
        return _state_of(s)
    _release(s, s["low"])
    _compact(s, c)
    _reserve(s, s["low"], c["len"], c)
    _release(s, s["high"])
    _compact(s, c)
    _reserve(s, s["high"], c["len"], c)
    return _state_of(s)


# ------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    """Attention sequence by sequence and row by row of the definition, in
    64 bits; written rows as their format's definition stores them (whose
    roundings are taken on fp32 values); page operators move bits."""
    c = dict(case)
    if c["op"] not in ("attention", "append"):
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    D, P, H = c["dim"], c["page"], c["heads"]
    lens, news = _lens(c), _news(c)
    layer = s["data"][c["layers"] - 1]

    def turned(x, p, t):
        """One row [heads, dim] rotated for position p, in type t."""
        x = x.to(t)
        if not c["rope"]:
            return x
        co, si = s["rope"][p, :, 0].to(t), s["rope"][p, :, 1].to(t)
        y = x.clone()
        r = c["rot"]
        a, b = (slice(0, r, 2), slice(1, r, 2)) if c["rope"] == 1 else (slice(0, r // 2), slice(r // 2, r))
        y[..., a] = x[..., a] * co - x[..., b] * si
        y[..., b] = x[..., b] * co + x[..., a] * si
        return y

    if c["op"] == "append":
        ks, vs = torch.zeros(s["k"].shape, dtype=f64, device="cuda"), torch.zeros(s["v"].shape, dtype=f64, device="cuda")
        for b in range(c["B"]):
            n = news[b]
            p = lens[b] + torch.arange(n, device="cuda")
            x = s["k"][b, :n]
            if c["rope"]:
                co, si = s["rope"][p][:, None, :, 0], s["rope"][p][:, None, :, 1]
                r = c["rot"]
                u, w = (slice(0, r, 2), slice(1, r, 2)) if c["rope"] == 1 else (slice(0, r // 2), slice(r // 2, r))
                y = x.clone()
                y[..., u] = x[..., u] * co - x[..., w] * si
                y[..., w] = x[..., w] * co + x[..., u] * si
                x = y
            for to, row in ((ks, x), (vs, s["v"][b, :n])):
                if c["type"] == "i8":
                    d = row.abs().max(-1, keepdim=True).values
                    d = d / torch.full_like(d, 127.0)
                    y = row * (1.0 / d)
                    y = torch.sign(y) * torch.floor(y.abs().double() + 0.5)
                    to[b, :n] = y.clamp(-127, 127) * d.double()
                else:
                    to[b, :n] = row.to(torch.float16 if c["type"] == "f16" else torch.bfloat16).to(f64)
        return ks, vs

    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    size = 1 if c["type"] == "i8" else 2
    t = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}[c["type"]]
    for b in range(c["B"]):
        n, new = lens[b], news[b]
        total = n + new
        masks = [(int(s["tree"][b, m]) if s["tree"] is not None else (2 << m) - 1) for m in range(new)]
        place = [n + bin(masks[m] & ((1 << m) - 1)).count("1") for m in range(new)]
        qs = torch.stack([turned(s["q"][b, m], place[m], f64) for m in range(new)])
        slot = torch.arange(total, device="cuda")
        at = slot.clone()
        at[n:] = torch.tensor(place, device="cuda")
        vis = torch.ones(new, total, dtype=torch.bool, device="cuda")
        for m in range(new):
            vis[m, n:] = torch.tensor([bool(masks[m] >> j & 1) for j in range(new)], device="cuda")
            if c["window"]:
                vis[m] &= (place[m] - at < c["window"]) | (at < c["sinks"])
        page = s["table"][b].long()[slot // P]
        for h in range(H):
            base = ((page * H + h) * (P // 32) + slot % P // 32) * _block_bytes(c)
            d = torch.arange(D, device="cuda")
            o = (slot % 32)[:, None]
            flat = layer.view(-1)
            k = flat.view(t)[(base // size)[:, None] + (d // 8 * 32 + o) * 8 + d % 8].to(f64)
            v = flat.view(t)[(base // size)[:, None] + 32 * D + (o // 8 * D + d) * 8 + o % 8].to(f64)
            if size == 1:
                f = flat.view(torch.float32)
                k *= f[base // 4 + 16 * D + slot % 32][:, None].to(f64)
                v *= f[base // 4 + 16 * D + 32 + slot % 32][:, None].to(f64)
            q = qs[:, h * c["group"]:(h + 1) * c["group"]]
            x = torch.tensordot(q, k, dims=([2], [1])) / math.sqrt(D)
            x = torch.where(vis[:, None, :], x, -math.inf)
            w = torch.softmax(x, -1)
            w = torch.where(vis[:, None, :].any(-1, keepdim=True), w, 0.0)
            out[b, :new, h * c["group"]:(h + 1) * c["group"]] = torch.tensordot(w, v, dims=([2], [0]))
    return out
