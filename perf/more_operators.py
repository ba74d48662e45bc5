"""Workloads of a round of several sequences that continue one prompt:
attention over a prefix that they share, the residual's addition with the RMS
norm and its int8 output, and sampling with temperature, top-k, top-p and
min-p.

Every case runs either in plain torch operations (own = False) or through
the package's calls (own = True) on the same buffers.

Layout of one cache block (32 positions of one head): keys [dim/8][32][8],
then values [4][dim][8] (8 positions innermost); int8 caches add 32 fp32
scales of the keys and 32 of the values.  A page holds its heads' blocks,
[heads][page/32]; the pool is [1][n_pages] pages.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f16": (1, torch.float16), "bf16": (30, torch.bfloat16), "i8": (24, torch.int8)}


# ------------------------------------------------------------------ cases
def listed():
    a = dict(op="attention", page=64, rot=128, rope=2, tree=False, ragged=True)
    s = dict(op="sample", sharp=2.0)
    n = dict(op="norm", delta=True, gamma=True)
    return [
        # four continuations of a short prompt, one token each: latency counts
        dict(a, name="shared_short", type="f16", B=4, M=1, heads=4, group=5, dim=128, prefix=1000, own=60),
        # plain sampling of 32 answers to one long prompt
        dict(a, name="shared_samples", type="bf16", B=32, M=1, heads=8, group=5, dim=128, prefix=16391, own=700),
        # verification rounds of 16 sequences that continue one document
        dict(a, name="shared_verify", type="f16", B=16, M=5, heads=8, group=5, dim=128, prefix=32768, own=1024),
        # draft trees of 8 sequences, int8 cache, large pages; adjacent-pair rotation of half of a head
        dict(a, name="shared_trees_i8", type="i8", B=8, M=16, heads=8, group=4, dim=64, prefix=8000, own=300, page=128,
             tree=True, rot=32, rope=1),
        # the next token of one sequence: latency counts
        dict(s, name="sample_one", rows=1, V=151936, filters="chat", probs=False, kept=False),
        # the rows of a verification round: distributions and filtered logits for rejection acceptance
        dict(s, name="sample_round", rows=5, V=151936, filters="nucleus", probs=True, kept=True),
        # drafts of a batch from a restricted head of 32768 + 256 tokens, with the distributions they are drawn from
        dict(s, name="sample_drafts", rows=48, V=33024, filters="nucleus", probs=True, kept=False),
        # the next tokens of a large batch, every row with settings of its own
        dict(s, name="sample_batch", rows=256, V=151936, filters="mixed", probs=False, kept=False),
        # the residual stream of one verification round: the norm's factor is left to the next projection
        dict(n, name="norm_round", rows=5, K=5120, fold=True, q8=True, y=False),
        # a batch's rounds, the vector and its codes
        dict(n, name="norm_batch", rows=80, K=2560, fold=False, q8=True, y=True),
        # a norm before a computation in fp32, odd row count
        dict(n, name="norm_plain", rows=3001, K=2560, fold=False, q8=False, y=True),
        # a prompt's rows
        dict(n, name="norm_prompt", rows=8192, K=5120, fold=False, q8=True, y=False),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "sample", "sample", "norm"])
    if op == "attention":
        c = dict(op=op, type=rng.choice(["f16", "bf16", "i8"]), B=_spread(rng, 2, 40), M=rng.choice([1, 1, 3, 5, 8, 16]),
                 heads=rng.choice([1, 2, 3, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 7, 8]),
                 dim=rng.choice([32, 64, 96, 128, 128, 160, 256]), page=rng.choice([32, 64, 128, 256]),
                 rope=rng.choice([0, 1, 2]), tree=rng.random() < 0.3, ragged=rng.random() < 0.7)
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2])
        rows = c["B"] * c["M"] * c["group"] * c["heads"]
        c["own"] = _spread(rng, 1, max(10, min(2000, (1 << 31) // (rows * c["dim"]))))
        c["prefix"] = _spread(rng, 40, max(60, min(60000, (1 << 33) // (rows * c["dim"]), (1 << 18) // c["heads"])))
        return c
    if op == "sample":
        V = _spread(rng, 30, 200000)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(400, 30000000 // V))), V=V, sharp=rng.choice([0.5, 1.0, 2.0, 3.0]),
                    filters=rng.choice(["chat", "nucleus", "mixed", "mixed", "none", "least"]), probs=rng.random() < 0.4,
                    kept=rng.random() < 0.3)
    K = 32 * _spread(rng, 1, 768)
    c = dict(op=op, K=K, rows=_spread(rng, 1, max(1, min(9000, 40000000 // K))), delta=rng.random() < 0.8,
             gamma=rng.random() < 0.8, fold=rng.random() < 0.4)
    c["q8"] = c["fold"] or rng.random() < 0.7
    c["y"] = not c["fold"] and (not c["q8"] or rng.random() < 0.5)
    return c


# ------------------------------------------------------- sizes of a case
def _some(c, most):
    """`most` for the first sequence, and for the others where the case is
    not ragged; else numbers spread over 1 .. most."""
    if not c["ragged"]:
        return [most] * c["B"]
    return [most if b == 0 else max(1, int(most * ((b * 0.6180339887) % 1.0))) for b in range(c["B"])]


def _lens(c):
    """Cached positions of each sequence: the prompt and its own ones."""
    return [c["prefix"] + n for n in _some(c, c["own"])]


def _shared(c):
    """Slots that lie in pages which the sequences share: the full ones."""
    return c["prefix"] // c["page"] * c["page"]


def _width(c):
    return -(-(c["prefix"] + c["own"] + c["M"]) // c["page"])


def _block_bytes(c):
    return 64 * c["dim"] + 256 if c["type"] == "i8" else 128 * c["dim"]


def _row_bytes(c):
    """Bytes of one position of one head: its key and its value."""
    return 2 * c["dim"] + 8 if c["type"] == "i8" else 4 * c["dim"]


def work(c):
    if c["op"] == "attention":
        lens, news = _lens(c), _some(c, c["M"])
        held = _shared(c) + sum(n + new - _shared(c) for n, new in zip(lens, news))
        pairs = sum((n + new) * new for n, new in zip(lens, news)) * c["heads"] * c["group"]
        qo = 2 * sum(news) * c["heads"] * c["group"] * c["dim"] * 4
        return {"bytes": held * c["heads"] * _row_bytes(c) + qo, "flops": 4.0 * pairs * c["dim"]}
    if c["op"] == "sample":
        n = c["rows"] * c["V"]
        return {"bytes": 4 * n * (1 + c["probs"] + c["kept"]) + 28 * c["rows"], "flops": 4.0 * n}
    n = c["rows"] * c["K"]
    return {"bytes": int(n * (8 + 4 * c["delta"] + 4 * c["y"] + (1 + 16 / 32) * c["q8"])) + 4 * c["K"] * c["gamma"],
            "flops": 8.0 * n}


# --------------------------------------------------------------- inputs
def _pool(c, n_pages, gen):
    """A pool whose every position holds a finite row."""
    page_bytes = c["heads"] * (c["page"] // 32) * _block_bytes(c)
    if c["type"] != "i8":
        x = torch.empty(n_pages, page_bytes // 2, dtype=TYPES[c["type"]][1], device="cuda")
        x.normal_(generator=gen)
        return x.view(torch.uint8).view(1, n_pages, page_bytes)
    blocks = n_pages * c["heads"] * (c["page"] // 32)
    x = torch.empty(blocks, _block_bytes(c), dtype=torch.uint8, device="cuda")
    codes = 64 * c["dim"]
    x[:, :codes] = torch.randint(-127, 128, (blocks, codes), device="cuda", generator=gen, dtype=torch.int8).view(torch.uint8)
    scale = 0.014 * (0.5 + torch.rand(blocks, 64, device="cuda", generator=gen))
    x[:, codes:] = scale.view(torch.uint8)
    return x.view(1, n_pages, page_bytes)


def _trees(c, seed):
    """A parent among the earlier rows for every row but the first; a row
    sees itself and its ancestors."""
    r = np.random.RandomState((seed * 1000003 + 17) % (1 << 31))
    masks = np.zeros((c["B"], c["M"]), np.int64)
    for b in range(c["B"]):
        for m in range(c["M"]):
            masks[b, m] = (1 << m) | (masks[b, r.randint(0, m)] if m else 0)
    return torch.from_numpy(masks.astype(np.int32)).cuda()


def _settings(c, seed):
    """(temperature, top_k, top_p, min_p) of every row, or one for all."""
    if c["filters"] == "chat":
        return [(0.8, 40, 0.95, 0.0)]
    if c["filters"] == "nucleus":
        return [(1.0, 0, 0.9, 0.02)]
    if c["filters"] == "none":
        return [(1.0, 0, 1.0, 0.0)]
    if c["filters"] == "least":
        return [(1.2, 0, 1.0, 0.05)]
    r = np.random.RandomState((seed * 1000003 + 29) % (1 << 31))
    rows = []
    for _ in range(c["rows"]):
        rows.append((float(r.choice([0.0, 0.3, 0.7, 1.0, 1.5])), int(r.choice([0, 0, 1, 20, 50, 500])),
                     float(r.choice([1.0, 0.5, 0.9, 0.95, 0.99])), float(r.choice([0.0, 0.0, 0.02, 0.1]))))
    return rows


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    s = {"case": c, "handle": None}
    if c["op"] == "attention":
        B, M, P, W, lens = c["B"], c["M"], c["page"], _width(c), _lens(c)
        full = c["prefix"] // P
        need = [-(-(n + M) // P) - full for n in lens]
        n_pages = full + sum(need) + 3
        s["data"] = _pool(c, n_pages, gen)
        order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
        ints = dict(dtype=torch.int32, device="cuda")
        s["table"] = torch.full((B, W), -1, **ints)
        s["table"][:, :full] = order[:full]
        s["refs"] = torch.zeros(n_pages, **ints)
        s["refs"][order[:full].long()] = B
        at = full
        for b, k in enumerate(need):
            s["table"][b, full:full + k] = order[at:at + k]
            s["refs"][order[at:at + k].long()] = 1
            at += k
        s["free_ids"] = torch.zeros(n_pages, **ints)
        s["free_ids"][:n_pages - at] = order[at:]
        s["ctl"] = torch.tensor([n_pages - at, 0, 0, 0], **ints)
        s["len"] = torch.tensor(lens, **ints)
        s["n_new"] = torch.tensor(_some(c, M), **ints) if c["ragged"] else None
        s["tree"] = _trees(c, seed) if c["tree"] else None
        s["rope"] = None
        if c["rope"]:   # cos and sin of every position's angles, in 64 bits and then rounded
            inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
            ang = torch.arange(W * P, dtype=torch.float64, device="cuda")[:, None] * inv
            s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        s["q"] = normal(B, M, c["heads"] * c["group"], c["dim"]) * 1.5
        s["out"] = torch.zeros_like(s["q"])
        return s
    if c["op"] == "sample":
        R, V = c["rows"], c["V"]
        # most tokens near each other, one in 64 above them with an exponential tail
        z = normal(R, V) * 1.5
        up = torch.rand(R, V, device="cuda", generator=gen) < 1 / 64
        z += torch.where(up, 3.0 + c["sharp"] * torch.empty_like(z).exponential_(generator=gen), 0.0)
        s["logits"] = z
        s["settings"] = np.array(_settings(c, seed), np.float64)
        s["u"] = torch.rand(R, dtype=torch.float64, device="cuda", generator=gen)
        s["tokens"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        s["probs"] = torch.zeros_like(z) if c["probs"] else None
        s["kept"] = torch.zeros_like(z) if c["kept"] else None
        temperature, top_k, top_p, min_p = s["settings"].T
        col = lambda x, t: torch.from_numpy(x.astype(t)).cuda()[:, None]  # noqa: E731
        s["columns"] = (col(temperature, np.float32).double(), col(top_k, np.int64), col(top_p, np.float32).double(),
                        col(min_p, np.float32).double())
        return s
    R, K = c["rows"], c["K"]
    s["x"] = normal(R, K) * 2.0
    s["x"][:, ::97] *= 20.0                        # a residual stream has a few large channels
    s["delta"] = normal(R, K) if c["delta"] else None
    s["gamma"] = 1.0 + 0.1 * normal(K) if c["gamma"] else None
    new = lambda t, *n: torch.zeros(*n, dtype=t, device="cuda")  # noqa: E731
    s["sum"] = new(torch.float32, R, K)
    s["y"] = new(torch.float32, R, K) if c["y"] else None
    s["values"] = None
    if c["q8"]:
        s["q"], s["d"], s["s16"] = new(torch.int8, R, K), new(torch.float32, R, K // 32), new(torch.int32, R, K // 16)
        s["sumsq"], s["values"] = new(torch.float32, R, K // 32), new(torch.float32, R, K)
    return s


# ------------------------------------------------------ the plain forms
def _slots(s, c, pages):
    """Keys and values of the pages [..., n] as fp32 [..., heads, n * page, dim]."""
    D, nb = c["dim"], c["page"] // 32
    x = s["data"][0][pages.clamp(min=0).long()]
    lead = pages.shape[:-1]
    x = x.view(*lead, pages.shape[-1], c["heads"], nb, _block_bytes(c))
    t = TYPES[c["type"]][1]
    half = 32 * D * (1 if t == torch.int8 else 2)
    k = x[..., :half].contiguous().view(t).view(*x.shape[:-1], D // 8, 32, 8).float()
    v = x[..., half:2 * half].contiguous().view(t).view(*x.shape[:-1], 4, D, 8).float()
    k = k.transpose(-3, -2).reshape(*x.shape[:-1], 32, D)
    v = v.transpose(-2, -1).reshape(*x.shape[:-1], 32, D)
    if t == torch.int8:
        d = x[..., 2 * half:].contiguous().view(torch.float32)
        k, v = k * d[..., :32, None], v * d[..., 32:, None]
    n = pages.shape[-1] * c["page"]
    return tuple(y.transpose(-5, -4).reshape(*lead, c["heads"], n, D) for y in (k, v))


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
    """The prefix for all rows in one product a head, each sequence's own
    slots for its rows, one softmax over both."""
    B, M, H, G, D = c["B"], c["M"], c["heads"], c["group"], c["dim"]
    full = c["prefix"] // c["page"]
    n = s["len"].long()
    new = s["n_new"].long() if s["n_new"] is not None else torch.full_like(n, M)
    m = torch.arange(M, device="cuda")
    if s["tree"] is not None:
        sees = ((s["tree"].long()[:, :, None] >> m) & 1).bool()
    else:
        sees = (m[None, :] <= m[:, None]).expand(B, M, M)
    pos = n[:, None] + (sees & (m[None, :] < m[:, None])).sum(-1)
    q = _rotate(s["q"], pos, s, c).view(B, M, H, G, D) / math.sqrt(D)
    k1, v1 = _slots(s, c, s["table"][:, full:])                        # [B, H, n, D]
    slot = full * c["page"] + torch.arange(k1.shape[2], device="cuda")
    t = slot[None, :] - n[:, None]
    fresh = (t >= 0) & (t < new[:, None])
    vis = (t < 0)[:, None, :] | (fresh[:, None, :] & torch.gather(sees, 2, t.clamp(0, M - 1)[:, None, :].expand(B, M, -1)))
    v1 = v1 * vis.any(1)[:, None, :, None]
    q1 = q.permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    x1 = torch.matmul(q1, k1.transpose(-1, -2)).view(B, H, M, G, -1).masked_fill(~vis[:, None, :, None, :], -math.inf)
    x1 = x1.view(B, H, M * G, -1)
    top = x1.amax(-1, keepdim=True)
    if full:
        k0, v0 = _slots(s, c, s["table"][0, :full])                    # [H, n, D]
        q0 = q.permute(2, 0, 1, 3, 4).reshape(H, B * M * G, D)
        x0 = torch.matmul(q0, k0.transpose(-1, -2))                    # [H, B * M * G, n]
        top0 = x0.amax(-1, keepdim=True).view(H, B, M * G, 1).transpose(0, 1)
        top = torch.maximum(top, top0)
        e0 = torch.exp(x0 - top.transpose(0, 1).reshape(H, B * M * G, 1))
    top = torch.where(top == -math.inf, 0.0, top)
    e1 = torch.exp(x1 - top)
    total, o = e1.sum(-1, keepdim=True), torch.matmul(e1, v1)
    if full:
        back = lambda y: y.view(H, B, M * G, -1).transpose(0, 1)  # noqa: E731
        total, o = total + back(e0.sum(-1, keepdim=True)), o + back(torch.matmul(e0, v0))
    o = (o / torch.where(total == 0, 1.0, total)).view(B, H, M, G, D).permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D)
    live = m[None, :] < new[:, None]
    s["out"].copy_(torch.where(live[:, :, None, None], o, s["out"]))
    return s["out"]


def _sample(s, c):
    """In 64 bits: a token next to a border of the running sum changes with
    the sum's last digits."""
    z = s["logits"].double()
    temperature, top_k, top_p, min_p = s["columns"]
    V = c["V"]
    greedy = temperature == 0
    top_k = torch.where(greedy, 1, torch.where(top_k == 0, V, top_k.clamp(max=V)))
    order, index = torch.sort(z, dim=-1, descending=True, stable=True)
    w = torch.exp((order - order[:, :1]) / torch.where(greedy, 1.0, temperature))
    keep = torch.arange(V, device="cuda") < top_k
    w = w * keep
    run_to = w.cumsum(-1)
    keep = keep & ((run_to - w < top_p * run_to[:, -1:]) | (top_p >= 1)) & (w >= min_p)
    keep[:, 0] = True
    w = torch.zeros_like(z).scatter_(-1, index, w * keep)
    mass = w.cumsum(-1)
    over = mass > s["u"][:, None] * mass[:, -1:]
    s["tokens"].copy_(over.to(torch.uint8).argmax(-1))
    if c["probs"]:
        s["probs"].copy_(w / mass[:, -1:])
    if c["kept"]:
        keep = torch.zeros_like(keep).scatter_(-1, index, keep)
        s["kept"].copy_(torch.where(keep, s["logits"], -math.inf))
    return [x for x in (s["tokens"], s["probs"], s["kept"]) if x is not None]


def _norm(s, c):
    R, K = c["rows"], c["K"]
    t = s["x"] + s["delta"] if c["delta"] else s["x"]
    s["sum"].copy_(t)
    v = t * s["gamma"] if c["gamma"] else t
    squares = (t * t).view(R, K // 32, 32).sum(-1)
    r = 1.0 / torch.sqrt(squares.sum(-1, keepdim=True) / K + 1e-6)
    if c["y"]:
        s["y"].copy_(v * r)
    if c["q8"]:
        v = v.view(R, K // 32, 32)
        full = torch.full((1,), 127.0, device="cuda")      # a tensor: torch would multiply by a number's reciprocal
        d = v.abs().amax(-1, keepdim=True) / full
        x = v * torch.where(d > 0, 1.0 / d, 0.0)
        low = x.abs().floor()
        code = torch.copysign(low + (x.abs() - low >= 0.5).float(), x).clamp(-127, 127)
        s["s16"].copy_(code.view(R, K // 16, 16).sum(-1))
        s["values"].copy_((code * (d if c["fold"] else d * r[..., None])).view(R, K))
        s["sumsq"].copy_(squares)
    return _norm_outputs(s)


def _norm_outputs(s):
    out = [s["sum"]]
    if s["y"] is not None:
        out.append(s["y"])
    if s["values"] is not None:
        out += [s["values"], s["s16"], s["sumsq"]]
    return out


# --------------------------------------------------------------- the pass
def _plan(s, c):
    """The package's cache object over the state's buffers, and the plan of
    its attention: made at the first pass, as a program makes them once."""
    import speculative_decoding_verification_amd as sv
    kv = sv.KvCache(TYPES[c["type"]][0], 1, c["heads"], c["dim"], c["page"], s["refs"].numel(), c["B"], _width(c),
                    buffers={k: s[k] for k in ("data", "table", "len", "refs", "free_ids", "ctl")})
    rope = sv.Rope(c["rope"], c["rot"], s["rope"]) if c["rope"] else None
    s["handle"] = kv.attention(c["heads"] * c["group"], c["B"], c["M"], shared=_shared(c)), rope
    return s["handle"]


def _settings_of(s, c):
    """The rows' settings as the package takes them, and a workspace."""
    import speculative_decoding_verification_amd as sv
    temperature, top_k, top_p, min_p = s["settings"].T
    s["handle"] = sv.sampling_params(temperature, top_k.astype(np.int64), top_p, min_p), sv.sample_workspace(c["rows"], c["V"])
    return s["handle"]


def run(s):
    c = s["case"]
    if not own:
        return {"attention": _attention, "sample": _sample, "norm": _norm}[c["op"]](s, c)
    import speculative_decoding_verification_amd as sv
    if c["op"] == "attention":
        plan, rope = s["handle"] or _plan(s, c)
        plan.run(0, s["q"], s["out"], n_new=s["n_new"], tree=s["tree"], rope=rope)
        return s["out"]
    if c["op"] == "sample":
        params, workspace = s["handle"] or _settings_of(s, c)
        sv.sample(s["logits"], params, s["u"], s["tokens"], workspace, probs=s["probs"], kept=s["kept"])
        return [x for x in (s["tokens"], s["probs"], s["kept"]) if x is not None]
    codes = {k: s[k] for k in ("q", "d", "s16", "sumsq")} if c["q8"] else {}
    sv.add_norm_q8(s["x"], s["delta"], gamma=s["gamma"], fold=c["fold"], sum=s["sum"], y=s["y"], **codes)
    if c["q8"]:   # the codes as the values that they stand for
        torch.mul(s["q"].view(c["rows"], -1, 32), s["d"][..., None], out=s["values"].view(c["rows"], -1, 32))
    return _norm_outputs(s)


# ------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    """Attention sequence by sequence and row by row of the definition;
    sampling row by row on the host; the norm in 64 bits, with the roundings
    that its sum and its int8 format are defined by taken on fp32 values."""
    c = dict(case)
    if c["op"] == "sample" and c["rows"] * c["V"] > 45000000:
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "attention":
        return _exact_attention(s, c)
    if c["op"] == "sample":
        z, u = s["logits"].cpu().numpy(), s["u"].cpu().numpy()
        tokens = np.zeros(c["rows"], np.int32)
        probs = np.zeros(z.shape) if c["probs"] else None
        kept = np.full(z.shape, -np.inf) if c["kept"] else None
        for i, row in enumerate(z):
            temperature, k, p, least = s["settings"][min(i, len(s["settings"]) - 1)]
            temperature, p, least = (float(np.float32(x)) for x in (temperature, p, least))
            if temperature == 0:
                temperature, k = 1.0, 1
            best = row.max()
            j = np.arange(c["V"])
            if 0 < k < c["V"]:
                border = np.partition(row, c["V"] - int(k))[c["V"] - int(k)]
                above = np.flatnonzero(row > border)
                j = np.sort(np.concatenate([above, np.flatnonzero(row == border)[:int(k) - above.size]]))
            w = np.exp((row[j].astype(np.float64) - float(best)) / temperature)
            if p < 1:
                by = np.lexsort((j, -row[j].astype(np.float64)))
                need = p * w.sum()
                n = int(np.searchsorted(np.cumsum(w[by]), need, side="left")) + 1
                stay = np.sort(by[:n])
                j, w = j[stay], w[stay]
            j, w = j[w >= least], w[w >= least]
            mass = np.cumsum(w)
            tokens[i] = j[np.flatnonzero(mass > u[i] * mass[-1])[0]]
            if probs is not None:
                probs[i, j] = w / mass[-1]
            if kept is not None:
                kept[i, j] = row[j]
        return [torch.from_numpy(x) for x in (tokens, probs, kept) if x is not None]
    R, K = c["rows"], c["K"]
    t = s["x"] if s["delta"] is None else s["x"] + s["delta"]
    v = t if s["gamma"] is None else t * s["gamma"]
    wide = s["x"].to(f64) if s["delta"] is None else s["x"].to(f64) + s["delta"].to(f64)
    mean = t.to(f64).square().mean(-1, keepdim=True)
    r = (mean + float(np.float32(1e-6))).rsqrt()
    out = [wide]
    if c["y"]:
        out.append(wide * (1.0 if s["gamma"] is None else s["gamma"].to(f64)) * r)
    if c["q8"]:
        b = v.view(R, K // 32, 32)
        d = b.abs().max(-1, keepdim=True).values
        d = d / torch.full_like(d, 127.0)
        x = b * torch.where(d != 0, 1.0 / d, 0.0)
        code = (torch.sign(x) * torch.floor(x.abs().to(f64) + 0.5)).clamp(-127, 127)
        scale = d.to(f64) if c["fold"] else d.to(f64) * r[..., None]
        out += [(code * scale).view(R, K), code.view(R, K // 16, 16).sum(-1).to(torch.int32),
                t.to(f64).square().view(R, K // 32, 32).sum(-1)]
    return out


def _exact_attention(s, c):
    f64 = torch.float64
    D, P, H = c["dim"], c["page"], c["heads"]
    t = TYPES[c["type"]][1]
    size = 1 if t == torch.int8 else 2
    flat = s["data"].view(-1)
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    d = torch.arange(D, device="cuda")
    for b, (n, new) in enumerate(zip(_lens(c), _some(c, c["M"]))):
        masks = [(int(s["tree"][b, m]) if c["tree"] else (2 << m) - 1) for m in range(new)]
        place = [n + bin(masks[m] & ((1 << m) - 1)).count("1") for m in range(new)]
        q = s["q"][b, :new].to(f64)
        if c["rope"]:
            r = c["rot"]
            u, w = (slice(0, r, 2), slice(1, r, 2)) if c["rope"] == 1 else (slice(0, r // 2), slice(r // 2, r))
            cs = s["rope"][place].to(f64)[:, None]
            x = q.clone()
            x[..., u] = q[..., u] * cs[..., 0] - q[..., w] * cs[..., 1]
            x[..., w] = q[..., w] * cs[..., 0] + q[..., u] * cs[..., 1]
            q = x
        slot = torch.arange(n + new, device="cuda")
        vis = torch.ones(new, n + new, dtype=torch.bool, device="cuda")
        vis[:, n:] = torch.tensor([[bool(masks[m] >> j & 1) for j in range(new)] for m in range(new)], device="cuda")
        page = s["table"][b].long()[slot // P]
        for h in range(H):
            base = ((page * H + h) * (P // 32) + slot % P // 32) * _block_bytes(c)
            o = (slot % 32)[:, None]
            k = flat.view(t)[(base // size)[:, None] + (d // 8 * 32 + o) * 8 + d % 8].to(f64)
            v = flat.view(t)[(base // size)[:, None] + 32 * D + (o // 8 * D + d) * 8 + o % 8].to(f64)
            if size == 1:
                f = flat.view(torch.float32)
                k *= f[base // 4 + 16 * D + slot % 32][:, None].to(f64)
                v *= f[base // 4 + 16 * D + 32 + slot % 32][:, None].to(f64)
            qh = q[:, h * c["group"]:(h + 1) * c["group"]].reshape(-1, D)
            x = torch.mm(qh, k.t()).view(new, c["group"], -1) / math.sqrt(D)
            x = torch.where(vis[:, None, :], x, -math.inf)
            w = torch.softmax(x, -1).view(new * c["group"], -1)
            out[b, :new, h * c["group"]:(h + 1) * c["group"]] = torch.mm(w, v).view(new, c["group"], D)
    return out
