"""Cases for what positions and drafted tokens add to a transformer layer held
in 8 bits: the norms of queries and keys per head with the position rotation
(and their gradient), the cache's append with both on the way, attention over a
tree of drafted tokens, their verification, and keeping the accepted ones.

`own` chooses what run() calls: the library's entry points, or the plain form
in elementary torch operations. An 8-bit code is returned as the E4M3 number it
stands for, a scale byte as the power of two it stands for.

Heads lie [tokens, heads, dim]; q, k and v are slices of one projection's rows.
A rotation turns pairs of the first `rot` dims, (i, i + rot / 2) or (2 i, 2 i +
1), by a table [length, rot] of cosines, then sines. The cache has pages of
E4M3 codes and one scale byte per page and head, keys [page, head, token, dim],
values [page, head, dim, token]. A sequence's drafted tokens are nodes of a
tree: node 0 is its last token, parents come before their children, and a row
of the mask has a bit for each node that a node sees (its ancestors, itself).
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
MOST_ELEMS = 4e7     # of a drawn rotation's heads
MOST_TABLE = 6.5e7   # probabilities of a drawn verification


def listed():
    return [
        # one decoding step of a small batch: the latency of q's and k's norms
        {"name": "rotate token", "op": "rotate", "tokens": 5, "seqs": 5, "q_heads": 32, "k_heads": 8,
         "dim": 128, "rot": 128, "paired": False, "norm": True, "dtype": "bf16", "length": 16384},
        # prompts' queries and keys in one pass
        {"name": "rotate prompt", "op": "rotate", "tokens": 8191, "seqs": 3, "q_heads": 32,
         "k_heads": 8, "dim": 128, "rot": 128, "paired": False, "norm": True, "dtype": "bf16",
         "length": 16384},
        # the same in training: gradients of q, k and both norms' weights
        {"name": "rotate gradient", "op": "rotate_grad", "tokens": 8192, "seqs": 4, "q_heads": 32,
         "k_heads": 8, "dim": 128, "rot": 128, "paired": False, "norm": True, "dtype": "bf16",
         "length": 16384},
        # one new token for each sequence of a serving batch
        {"name": "append token", "op": "append", "batch": 64, "new": 1, "held": 300, "heads": 8,
         "dim": 128, "page": 64, "rot": 128, "paired": False, "norm": True, "drafted": False,
         "dtype": "bf16", "ragged": 1},
        # prompts entering the cache, the first one behind a held prefix
        {"name": "append prompt", "op": "append", "batch": 6, "new": 8000, "held": 77, "heads": 8,
         "dim": 128, "page": 64, "rot": 128, "paired": False, "norm": True, "drafted": False,
         "dtype": "bf16", "ragged": 2},
        # a few drafted tokens of short chats, latency counts
        {"name": "tree short", "op": "attend", "batch": 2, "new": 8, "context": 700, "heads": 8,
         "group": 4, "dim": 64, "page": 32, "chain": False, "ragged": 3},
        # a serving batch's trees over long contexts: the cache is read once
        {"name": "tree long", "op": "attend", "batch": 16, "new": 24, "context": 32000, "heads": 8,
         "group": 4, "dim": 128, "page": 64, "chain": False, "ragged": 4},
        # wide trees, many query heads to a kv head
        {"name": "tree wide", "op": "attend", "batch": 4, "new": 63, "context": 8000, "heads": 4,
         "group": 8, "dim": 128, "page": 64, "chain": False, "ragged": 5},
        # a tree that a greedy draft proposed (no probabilities of its own), one sequence
        {"name": "verify tree", "op": "verify", "batch": 1, "new": 12, "vocab": 32001,
         "draft": False, "chain": False, "dtype": "f32", "ragged": 6},
        # a serving batch's chains of drafted tokens with the draft's probabilities
        {"name": "verify chains", "op": "verify", "batch": 64, "new": 8, "vocab": 128000,
         "draft": True, "chain": True, "dtype": "f32", "ragged": 7},
        # the accepted tokens of one sequence
        {"name": "keep one", "op": "keep", "batch": 1, "new": 8, "held": 700, "heads": 8, "dim": 64,
         "page": 32, "ragged": 8},
        # those of a serving batch's trees
        {"name": "keep batch", "op": "keep", "batch": 64, "new": 32, "held": 3000, "heads": 8,
         "dim": 128, "page": 64, "ragged": 9},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotate", "rotate", "rotate_grad", "append", "append", "attend", "attend",
                     "attend", "verify", "verify", "keep"])
    if op in ("rotate", "rotate_grad"):
        dim, k_heads = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8])
        q_heads = k_heads * rng.choice([1, 2, 4, 5])
        most = max(1, min(8192, int(MOST_ELEMS / (dim * (q_heads + k_heads)))))
        tokens = spread(1, most)
        return {"op": op, "tokens": tokens, "seqs": min(tokens, spread(1, 64)), "q_heads": q_heads,
                "k_heads": k_heads, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim // 4]),
                "paired": rng.random() < 0.4, "norm": rng.random() < 0.7,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "length": spread(9000, 40000)}
    if op == "verify":
        vocab, draft = spread(1000, 130000), rng.random() < 0.6
        new = spread(1, 24)
        most = MOST_TABLE / vocab / new
        return {"op": op, "batch": max(1, min(64, spread(1, max(1, int(most))))), "new": new,
                "vocab": vocab, "draft": draft, "chain": rng.random() < 0.5,
                "dtype": rng.choice(["f32", "f32", "bf16"]), "ragged": rng.randrange(1 << 20)}
    heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([32, 64, 128])
    ragged = rng.randrange(1 << 20)
    if op == "append":
        batch, new = spread(1, 64), rng.choice([1, 1, spread(2, 64), spread(2, 4000)])
        new = min(new, max(1, 48000 // batch))
        return {"op": op, "batch": batch, "new": new, "held": spread(1, 1000), "heads": heads,
                "dim": dim, "page": page, "rot": rng.choice([dim, dim, dim // 2, dim // 4]),
                "paired": rng.random() < 0.4, "norm": rng.random() < 0.7,
                "drafted": new <= 64 and rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "ragged": ragged}
    if op == "keep":
        return {"op": op, "batch": spread(1, 64), "new": spread(2, 64), "held": spread(1, 4000),
                "heads": heads, "dim": dim, "page": page, "ragged": ragged}
    batch, new = spread(1, 32), spread(1, 64)
    return {"op": op, "batch": batch, "new": new,
            "context": new + spread(16, min(32000, 500000 // batch)), "heads": heads,
            "group": rng.choice([1, 2, 3, 4, 6, 8]), "dim": dim, "page": page,
            "chain": rng.random() < 0.3, "ragged": ragged}


def lengths(case):
    """(new tokens, tokens in the cache) of each sequence: for append and keep the
    tokens held before, for attend the tokens to read, the new ones among them. The
    first sequence is the longest; the last of four or more is an idle slot."""
    r, new, held = random.Random(case["ragged"]), [], []
    for i in range(case["batch"]):
        n = case["new"] if i == 0 else r.randint((case["new"] + 1) // 2, case["new"])
        if case["op"] == "attend":
            h = case["context"] if i == 0 else r.randint(max(n, case["context"] // 4),
                                                         max(n, case["context"]))
        else:
            h = r.randint(0, case.get("held", 0)) if i else case.get("held", 0)
        if i == case["batch"] - 1 >= 3:
            n = 0
        new.append(n)
        held.append(h)
    return new, held


def trees(case, new):
    """Each sequence's parents, node by node."""
    r = random.Random(case["ragged"] + 1)
    return [[-1 if j == 0 else j - 1 if case["chain"] else r.randint(max(0, j - 4), j - 1)
             for j in range(n)] for n in new]


def seen_by(parents):
    """Each node's ancestors and itself, as the bits of a whole number."""
    bits = []
    for j, p in enumerate(parents):
        bits.append(1 << j | (bits[p] if p >= 0 else 0))
    return bits


def numbers(shape, g, dtype=torch.bfloat16, by=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * by).to(dtype)


def whole(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def random_codes(shape, g):
    """E4M3 codes of normal values whose blocks' largest lie near the top of the range."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        x = torch.randn(part.shape, generator=g, device="cuda").mul_(100).clamp_(-448, 448)
        part.copy_(x.to(F8).view(torch.uint8))
    return out


def random_scales(shape, g):
    return torch.randint(118, 122, shape, generator=g, device="cuda", dtype=torch.uint8)


def rotary_table(length, rot):
    """Cosines, then sines, of every position's angles."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def weights(case, g, dtype):
    return numbers((case["dim"],), g, torch.float32, 0.2).add_(1).to(dtype) if case["norm"] else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("rotate", "rotate_grad"):
        dt, tokens, hq, hk = DTYPES[case["dtype"]], case["tokens"], case["q_heads"], case["k_heads"]
        qkv = numbers((tokens, hq + 2 * hk, case["dim"]), g, dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"], s["k_weight"] = weights(case, g, dt), weights(case, g, dt)
        s["table"] = rotary_table(case["length"], case["rot"])
        seq = torch.arange(tokens, device="cuda") * case["seqs"] // tokens
        first = -(-torch.arange(case["seqs"], device="cuda") * tokens // case["seqs"])
        start = torch.randint(0, case["length"] - 8192, (case["seqs"],), generator=g, device="cuda")
        s["positions"] = (start[seq] + torch.arange(tokens, device="cuda") - first[seq]).int()
        if op == "rotate_grad":
            s["dq"] = numbers((tokens, hq, case["dim"]), g, dt, 0.01)
            s["dk"] = numbers((tokens, hk, case["dim"]), g, dt, 0.01)
        return s
    new, held = lengths(case)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = whole(cu)
    if op == "verify":
        return prepare_verify(case, s, new, cu, g)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    total = [h if op == "attend" else n + h for n, h in zip(new, held)]
    pages = [-(-t // page) for t in total]
    pool = sum(pages) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["batch"], max(1, max(pages))), dtype=torch.int32, device="cuda")
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    s["cache"] = (random_codes((pool, heads, page, dim), g), random_scales((pool, heads), g),
                  random_codes((pool, heads, dim, page), g), random_scales((pool, heads), g))
    s["pages"], s["held"] = table, whole(held)
    s["most_new"], s["longest"] = max(new), max(total)
    if op == "append":
        dt = DTYPES[case["dtype"]]
        qkv = numbers((cu[-1], 3 * heads, dim), g, dt)
        s["k"], s["v"] = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
        s["weight"] = weights(case, g, dt)
        s["table"] = rotary_table(s["longest"], case["rot"])
        # a drafted token's position is its depth in the tree (here two to a depth)
        s["positions"] = whole([h + (j + 1) // 2 for n, h in zip(new, held) for j in range(n)]) \
            if case["drafted"] else None
    elif op == "attend":
        s["q"] = numbers((cu[-1], heads * case["group"], dim), g)
        words = -(-max(new) // 32)
        rows = [b >> 32 * w & 0xFFFFFFFF for p in trees(case, new) for b in seen_by(p)
                for w in range(words)]
        s["mask"] = whole([x - (1 << 32) if x >> 31 else x for x in rows]).view(cu[-1], words)
    else:
        r, most = random.Random(seed), max(1, min(case["new"], 9))
        path = []
        for n in new:
            some = sorted(r.sample(range(1, n), r.randint(0, min(n - 1, most - 1)))) if n else []
            path.append(([0] + some if n else []) + [-1] * (most - len(some) - (n > 0)))
        s["path"] = whole(path)
        s["count"] = (s["path"] >= 0).sum(1, dtype=torch.int32)
    return s


def prepare_verify(case, s, new, cu, g):
    """Probabilities as a language model has them: a few likely tokens, the draft's
    near the target's; drafted tokens drawn from the draft's."""
    rows, vocab, dt = cu[-1], case["vocab"], DTYPES[case["dtype"]]
    logits = torch.randn((rows, vocab), generator=g, device="cuda").mul_(3.5)
    s["target"] = torch.softmax(logits, 1).to(dt)
    logits.add_(torch.randn((rows, vocab), generator=g, device="cuda").mul_(0.7))
    draft = torch.softmax(logits, 1)
    del logits
    picks = torch.multinomial(draft, 4, replacement=True, generator=g)
    s["draft"] = draft.to(dt) if case["draft"] else None
    parents, parent_row, rank = [], [], []
    for p, at in zip(trees(case, new), cu):
        had = {}
        for j in p:
            had[j] = had.get(j, -1) + 1
            rank.append(had[j] % 4)
            parent_row.append(at + max(j, 0))
        parents += p
    s["parents"] = whole(parents)
    s["ids"] = picks[torch.tensor(parent_row, device="cuda"),
                     torch.tensor(rank, device="cuda")].to(torch.int32)
    s["numbers"] = torch.rand((rows, 2), generator=g, device="cuda")
    # what the tree's attention needed, too: which nodes a node sees
    bits = [[b >> j & 1 for j in range(case["new"])] for p in trees(case, new) for b in seen_by(p)]
    s["sees"] = torch.tensor(bits, dtype=torch.bool, device="cuda").view(rows, case["new"])
    s["width"] = max([b.bit_count() if hasattr(b, "bit_count") else bin(b).count("1")
                      for p in trees(case, new) for b in seen_by(p)])
    return s


def work(case):
    op = case["op"]
    if op in ("rotate", "rotate_grad"):
        e, both = 2 if case["dtype"] == "bf16" else 4, case["q_heads"] + case["k_heads"]
        n = case["tokens"] * both * case["dim"]
        if op == "rotate":
            return {"bytes": 2 * e * n + 4 * case["tokens"] * case["rot"], "flops": 8 * n}
        return {"bytes": e * n * (3 if case["norm"] else 2) + 4 * case["tokens"] * case["rot"],
                "flops": 16 * n}
    new, held = lengths(case)
    if op == "verify":
        # one row of each live sequence, the drafted tokens' probabilities
        e, live = 2 if case["dtype"] == "bf16" else 4, sum(n > 0 for n in new)
        return {"bytes": live * case["vocab"] * e * (2 if case["draft"] else 1) + 16 * sum(new),
                "flops": 2 * live * case["vocab"]}
    heads, dim = case["heads"], case["dim"]
    if op == "append":
        t, e = sum(new), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * t * heads * dim * (e + 1) + 4 * t * case["rot"],
                "flops": 12 * t * heads * dim}
    if op == "keep":
        moved = sum(n > 0 for n in new) * max(1, min(case["new"], 9)) // 2
        return {"bytes": 4 * max(1, moved) * heads * dim, "flops": 2 * max(1, moved) * heads * dim}
    pairs = sum(n * (h - n) + sum(bin(b).count("1") for b in seen_by(p))
                for n, h, p in zip(new, held, trees(case, new)))
    rows = sum(new) * heads * case["group"]
    return {"bytes": 2 * sum(h for n, h in zip(new, held) if n) * heads * dim + 4 * rows * dim,
            "flops": 4 * pairs * heads * case["group"] * dim}


# ---- the plain forms ----------------------------------------------------------

def plain_byte(amax):
    """Scale bytes of blocks with these largest magnitudes."""
    e = torch.frexp(amax).exponent.to(torch.int32) - 1
    return torch.where(amax > 0, (e - 8 + 127).clamp(0, 254), 0)


def power(e):
    """2^e of whole e, exactly (through the exponent field; at least 2^-126)."""
    return ((e.to(torch.int32) + 127).clamp(1, 254) << 23).view(torch.float32)


def plain_code(x, byte):
    """E4M3 of x / 2^(byte-127)."""
    return (x * power(127 - byte)).clamp(-448, 448).to(F8)


def pairs_of(x, paired):
    """The two members of each rotated pair."""
    if paired:
        return x[..., 0::2], x[..., 1::2]
    half = x.shape[-1] // 2
    return x[..., :half], x[..., half:]


def joined(a, b, paired):
    return torch.stack([a, b], -1).flatten(-2) if paired else torch.cat([a, b], -1)


def plain_turn(x, s, positions, sign=1.0):
    """x [tokens, heads, dim] rotated by its positions' angles, or back."""
    c = s["case"]
    cos, sin = s["table"].to(x.dtype)[positions.long()].unsqueeze(1).chunk(2, 2)
    sin = sin * sign
    a, b = pairs_of(x[..., :c["rot"]], c["paired"])
    turned = joined(a * cos - b * sin, b * cos + a * sin, c["paired"])
    return torch.cat([turned, x[..., c["rot"]:]], 2)


def plain_heads(x, weight, s, positions):
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * weight.to(x.dtype)
    return plain_turn(x, s, positions)


def plain_rotate(s):
    return {n: plain_heads(s[n].float(), s[n + "_weight"], s, s["positions"]).to(s[n].dtype)
            for n in ("q", "k")}


def plain_rotate_grad(s):
    out = {}

    def one(n):
        x, weight = s[n].float(), s[n + "_weight"]
        dn = plain_turn(s["d" + n].float(), s, s["positions"], -1.0)
        if weight is None:
            return dn.to(s[n].dtype)
        r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
        g = dn * weight.float()
        out["d" + n + "_weight"] = (dn * x * r).sum((0, 1))
        return (r * (g - x * (r * r) * (g * x).mean(2, keepdim=True))).to(s[n].dtype)

    out["dq"], out["dk"] = one("q"), one("k")
    return out


def plain_append(s):
    page, (cu, held, table) = s["case"]["page"], (s["cu"].long(), s["held"].long(), s["pages"].long())
    token = torch.arange(s["k"].shape[0], device=held.device)
    at = torch.searchsorted(cu[1:], token, right=True)
    positions = held[at] + token - cu[at] if s["positions"] is None else s["positions"]
    # a page's byte changes where its largest number crosses a power of two: 64 bits
    k = plain_heads(s["k"].double(), s["weight"], s, positions).float()
    new = cu[1:] - cu[:-1]
    steps = -(-s["most_new"] // page) + 1  # pages a sequence's new tokens can touch
    at = (held // page)[:, None] + torch.arange(steps, device=held.device)
    seq, j = torch.nonzero(at * page < (held + new)[:, None] * (new > 0)[:, None], as_tuple=True)
    at = at[seq, j]
    ids = table[seq, at]
    pos = at[:, None] * page + torch.arange(page, device=held.device)
    old = pos < held[seq][:, None]
    fresh = ~old & (pos < (held + new)[seq][:, None])
    src = (cu[seq][:, None] + pos - held[seq][:, None]).clamp(0, max(0, k.shape[0] - 1))

    def put(codes, scales, x, turn):
        v = x[src].permute(0, 2, 1, 3)                                # [n, head, token, dim]
        was = codes[ids].transpose(2, 3) if turn else codes[ids]
        f, o = fresh[:, None, :, None], old[:, None, :, None]
        byte = plain_byte((v * f).abs().amax((2, 3)))
        before = torch.where(old.any(1)[:, None], scales[ids].int(), 0)
        byte = torch.maximum(byte, before)
        b4 = byte[:, :, None, None]
        moved = (was.view(F8).float() * power(before[:, :, None, None] - b4)).to(F8)
        code = torch.where(f, plain_code(v, b4).view(torch.uint8),
                           torch.where(o, moved.view(torch.uint8), was))
        codes[ids] = code.transpose(2, 3) if turn else code
        scales[ids] = byte.to(torch.uint8)

    put(*s["cache"][:2], k, False)
    put(*s["cache"][2:], s["v"].float(), True)
    return cache_values(s)


def cache_values(s):
    k, ks, v, vs = s["cache"]
    return {"k": k.view(F8), "k_scales": ks.view(E8), "v": v.view(F8), "v_scales": vs.view(E8)}


def plain_attend(s):
    c, (k, ks, v, vs), q = s["case"], s["cache"], s["q"]
    cu, held, table = s["cu"].long(), s["held"].long(), s["pages"].long()
    batch, heads, group, dim = c["batch"], c["heads"], c["group"], c["dim"]

    def value(codes, scales):
        return codes[table].view(F8).float() * power(scales[table].int() - 127)[..., None, None]

    kd = value(k, ks).permute(0, 2, 1, 3, 4).reshape(batch, heads, -1, dim)
    vd = value(v, vs).permute(0, 2, 1, 4, 3).reshape(batch, heads, -1, dim)
    new, steps = cu[1:] - cu[:-1], torch.arange(s["most_new"], device=q.device)
    row = (cu[:-1, None] + steps).clamp(max=q.shape[0] - 1)
    qd = q.float()[row].view(batch, -1, heads, group, dim).permute(0, 2, 1, 3, 4)
    scores = qd.reshape(batch, heads, -1, dim) @ kd.transpose(2, 3)
    scores = scores.view(batch, heads, s["most_new"], group, -1) * (1.0 / math.sqrt(dim))
    # keys before the new tokens, and those new ones whose bit is set
    node = torch.arange(kd.shape[2], device=q.device) - (held - new)[:, None]
    word = s["mask"].long()[row].gather(2, (node >> 5).clamp(0, s["mask"].shape[1] - 1)
                                        .unsqueeze(1).expand(-1, s["most_new"], -1))
    bit = (word >> (node & 31).unsqueeze(1) & 1).bool() & (node < new[:, None]).unsqueeze(1)
    seen = (node < 0).unsqueeze(1) | bit
    scores = scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(4, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0, top)).exp_()
    total = p.sum(4, keepdim=True)
    o = p.view(batch, heads, -1, p.shape[4]) @ vd
    o = o.view(batch, heads, -1, group, dim) / torch.where(total == 0, 1, total)
    token = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu[1:], token, right=True)
    return o.permute(0, 2, 1, 3, 4)[seq, token - cu[seq]].reshape(q.shape).to(q.dtype)


def plain_verify(s):
    cu, parents, ids, p = s["cu"].long(), s["parents"].long(), s["ids"].long(), s["target"].double()
    rows, vocab = p.shape
    token = torch.arange(rows, device=p.device)
    seq = torch.searchsorted(cu[1:], token, right=True)
    child = parents >= 0
    up = torch.where(child, cu[seq] + parents, token)                 # a node's parent's row
    # each node's first child, and whether it is taken at once
    none = rows
    first = torch.full((rows,), none, device=p.device).scatter_reduce_(
        0, up, torch.where(child, token, none), "amin")
    has = first < none
    at = ids[first.clamp(max=rows - 1)]
    taken, w = torch.zeros_like(has), p
    if s["draft"] is not None:
        q, u = s["draft"].double(), s["numbers"][:, 0].double()
        taken = has & (u * q[token, at] < p[token, at])
        w = torch.where(has[:, None], (p - q).clamp(min=0), p)
        w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    # sums next to a border decide: 64 bits
    sums = w.cumsum(1)
    t = torch.searchsorted(sums, s["numbers"][:, 1:].double() * sums[:, -1:], right=True)[:, 0]
    last = torch.where(w > 0, torch.arange(vocab, device=p.device), -1).amax(1)
    t = torch.minimum(t, last)
    # the child that a node goes on to: the first one taken, or the first with the token
    goes = torch.where(taken[up], token == first[up], child & (ids == t[up]))
    on = torch.full((rows,), none, device=p.device).scatter_reduce_(
        0, up, torch.where(goes & child, token, none), "amin")
    followed = child & (on[up] == token)
    # a node is on the path where every one that it sees but the root was followed
    batch, n = cu.numel() - 1, s["sees"].shape[1]
    node = token - cu[seq]
    grid = torch.zeros((batch, n), dtype=torch.bool, device=p.device)
    grid[seq, node] = followed | (node == 0)
    path = ~(s["sees"] & ~grid[seq]).any(1)
    on_path = torch.zeros_like(grid)
    on_path[seq, node] = path
    count = on_path.sum(1)
    order = torch.where(on_path, torch.arange(n, device=p.device), n).sort(1).values[:, :s["width"]]
    end = (cu[:-1] + order.gather(1, (count[:, None] - 1).clamp(min=0))[:, 0]).clamp(max=rows - 1)
    return {"path": torch.where(order < n, order, -1).int(), "count": count.int(),
            "token": torch.where(count > 0, t[end], -1).int()}


def plain_keep(s):
    page, held, table = s["case"]["page"], s["held"].long(), s["pages"].long()
    path, count = s["path"].long(), s["count"].long()
    batch, width = path.shape
    step = torch.arange(width, device=held.device)
    live = step < count[:, None]
    stays = (path == step).long().cumprod(1).sum(1)                    # nodes that are in place
    # every page that an accepted token moves to
    near = -(-width // page) + 1
    at = (held // page)[:, None] + torch.arange(near, device=held.device)
    lo, hi = (held + stays)[:, None], (held + count)[:, None]
    seq, j = torch.nonzero(torch.maximum(at * page, lo) < torch.minimum((at + 1) * page, hi), as_tuple=True)
    at = at[seq, j]
    ids = table[seq, at]
    pos = at[:, None] * page + torch.arange(page, device=held.device)
    node = (pos - held[seq][:, None])
    fresh = (pos >= (held + stays)[seq][:, None]) & (pos < (held + count)[seq][:, None])
    old = pos < (held + stays)[seq][:, None]
    src = held[seq][:, None] + path[seq].gather(1, node.clamp(0, width - 1))
    src = torch.where(fresh, src, pos)
    from_page = table[seq][torch.arange(seq.numel(), device=held.device)[:, None],
                           (src // page).clamp(max=table.shape[1] - 1)]
    slot = src % page

    def move(codes, scales, turn):
        f, o = fresh[:, None, :, None], old[:, None, :, None]
        if turn:
            came = codes[from_page, :, :, slot].permute(0, 2, 1, 3)    # [n, head, token, dim]
            was = codes[ids].transpose(2, 3)
        else:
            came = codes[from_page, :, slot].permute(0, 2, 1, 3)
            was = codes[ids]
        s_came = scales[from_page].permute(0, 2, 1).int()              # [n, head, token]
        before = torch.where(old.any(1)[:, None], scales[ids].int(), 0)
        byte = torch.maximum(before, torch.where(fresh[:, None], s_came, 0).amax(2))
        b4 = byte[:, :, None, None]

        def rounded(code, by):
            return (code.contiguous().view(F8).float() * power(by - b4)).to(F8).view(torch.uint8)

        code = torch.where(f, rounded(came, s_came[..., None]),
                           torch.where(o, rounded(was, before[:, :, None, None]), was))
        return code.transpose(2, 3) if turn else code, byte.to(torch.uint8)

    k, ks, v, vs = s["cache"]
    new_k, new_v = move(k, ks, False), move(v, vs, True)
    k[ids], ks[ids] = new_k
    v[ids], vs[ids] = new_v
    return cache_values(s)


PLAIN = {"rotate": plain_rotate, "rotate_grad": plain_rotate_grad, "append": plain_append,
         "attend": plain_attend, "verify": plain_verify, "keep": plain_keep}


# ---- the library's calls -------------------------------------------------------

def rotary_of(s):
    import microscaling_fp4_block_mx_amd as mx
    return mx.Rotary(s["table"], s["positions"], s["case"]["paired"])


def own_rotate(s):
    import microscaling_fp4_block_mx_amd as mx
    q, k = mx.norm_rotate(s["q"], s["k"], s["q_weight"], s["k_weight"], rotary_of(s), EPS)
    return {"q": q, "k": k}


def own_rotate_grad(s):
    import microscaling_fp4_block_mx_amd as mx
    dq, dk, dq_weight, dk_weight = mx.norm_rotate_backward(
        s["dq"], s["q"], s["dk"], s["k"], s["q_weight"], s["k_weight"], rotary_of(s), EPS)
    out = {"dq": dq, "dk": dk}
    if s["case"]["norm"]:
        out["dq_weight"], out["dk_weight"] = dq_weight, dk_weight
    return out


def own_append(s):
    import microscaling_fp4_block_mx_amd as mx
    mx.kv_append_rotary(mx.KVCache(*s["cache"]), s["k"], s["v"], s["pages"], s["cu"], s["held"],
                        rotary_of(s), s["weight"], EPS)
    return cache_values(s)


def own_attend(s):
    import microscaling_fp4_block_mx_amd as mx
    return mx.kv_attention_tree(s["q"], mx.KVCache(*s["cache"]), s["pages"], s["cu"], s["held"],
                                s["mask"], max_length=s["longest"])


def own_verify(s):
    import microscaling_fp4_block_mx_amd as mx
    path, count, token = mx.verify_drafts(s["target"], s["ids"], s["parents"], s["cu"],
                                          s["numbers"], s["width"], draft=s["draft"])
    return {"path": path, "count": count, "token": token}


def own_keep(s):
    import microscaling_fp4_block_mx_amd as mx
    mx.kv_keep(mx.KVCache(*s["cache"]), s["pages"], s["held"], s["path"], s["count"])
    return cache_values(s)


OWN = {"rotate": own_rotate, "rotate_grad": own_rotate_grad, "append": own_append,
       "attend": own_attend, "verify": own_verify, "keep": own_keep}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---- 64 bits --------------------------------------------------------------------
# An 8-bit output's value is the number before its rounding to 8 bits, as a bf16
# output's is the number before its rounding to bf16.

def byte64(amax):
    s = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    s = torch.where(amax < torch.exp2(s), s - 1, s)
    s = torch.where(amax >= torch.exp2(s + 1), s + 1, s)
    return torch.where(amax > 0, (s + 119).clamp(0, 254), 0.0)


def turns64(s, positions):
    """[tokens, dim, dim]: each token's rotation, as a matrix applied from the left."""
    c, n = s["case"], positions.numel()
    half, dim = c["rot"] // 2, c["dim"]
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if c["paired"] else (i, i + half)
    row = s["table"].double()[positions.long()]
    m = torch.eye(dim, dtype=torch.float64, device="cuda").repeat(n, 1, 1)
    m[:, a, a] = row[:, :half]
    m[:, b, b] = row[:, :half]
    m[:, a, b] = -row[:, half:]
    m[:, b, a] = row[:, half:]
    return m


def apart(tokens, f):
    """f over runs of tokens that fit, joined."""
    return torch.cat([f(slice(i, min(tokens, i + 1024))) for i in range(0, tokens, 1024)])


def heads64(x, weight, s, positions):
    def part(at):
        y = x[at].double()
        if weight is not None:
            y = weight.double() * y / torch.sqrt(y.square().sum(2, keepdim=True) / x.shape[2] + EPS)
        return torch.bmm(y, turns64(s, positions[at]).transpose(1, 2).contiguous())
    return apart(x.shape[0], part)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rotate":
        return {n: heads64(s[n], s[n + "_weight"], s, s["positions"]) for n in ("q", "k")}
    if op == "rotate_grad":
        out = {}
        for n in ("q", "k"):
            x, w = s[n].double(), s[n + "_weight"]
            # the rotation's transpose, from the right
            dn = apart(x.shape[0], lambda at: torch.bmm(s["d" + n][at].double(),
                                                        turns64(s, s["positions"][at])))
            if w is None:
                out["d" + n] = dn
                continue
            root = torch.sqrt(x.square().sum(2, keepdim=True) / case["dim"] + EPS)
            unit, g = x / root, dn * w.double()
            out["d" + n] = (g - unit * (g * unit).sum(2, keepdim=True) / case["dim"]) / root
            out["d" + n + "_weight"] = (dn * unit).sum((0, 1))
        return out
    if op == "verify":
        return None
    new, held = lengths(case)
    page = case["page"]
    if op in ("append", "keep"):
        kc, ks, vc, vs = s["cache"]
        out = {"k": kc.view(F8).double(), "k_scales": torch.exp2(ks.double() - 127),
               "v": vc.view(F8).double().transpose(2, 3).contiguous(),
               "v_scales": torch.exp2(vs.double() - 127)}
        at = 0
        for i, (n, h) in enumerate(zip(new, held)):
            if not n:
                continue
            if op == "append":
                pos = s["positions"][at:at + n] if case["drafted"] else torch.arange(h, h + n, device="cuda")
                x = {"k": heads64(s["k"][at:at + n], s["weight"], s, pos), "v": s["v"][at:at + n].double()}
                place(out, s["pages"][i], page, h, x, None)
            else:
                path = s["path"][i].tolist()
                path = [p for p in path if p >= 0]
                stay = 0
                while stay < len(path) and path[stay] == stay:
                    stay += 1
                x, units = {}, {}
                ids = s["pages"][i].long()
                src = torch.tensor([h + p for p in path[stay:]], dtype=torch.int64, device="cuda")
                for name in ("k", "v"):
                    units[name] = out[name + "_scales"][ids[src // page]].clone()
                    x[name] = out[name][ids[src // page], :, src % page] * units[name][..., None]
                if len(path) > stay:
                    place(out, s["pages"][i], page, h + stay, x, units)
            at += n
        out["v"] = out["v"].transpose(2, 3).contiguous()
        return out
    return attend64(s, new, held)


def place(out, pages, page, h, x, units):
    """Puts x's tokens at positions h on; a page's unit is its kept tokens' or what
    the new ones need (`units`: what each came with), whichever is larger."""
    n = x["k"].shape[0]
    for j in range(h // page, -(-(h + n) // page)):
        p = int(pages[j])
        lo, hi = max(h, j * page), min(h + n, (j + 1) * page)
        kept, end = lo - j * page, hi - j * page
        for name in ("k", "v"):
            part = x[name][lo - h:hi - h].transpose(0, 1)
            unit = torch.exp2(byte64(part.abs().amax((1, 2))) - 127) if units is None \
                else units[name][lo - h:hi - h].amax(0)
            if kept:
                was = out[name + "_scales"][p].clone()
                unit = torch.maximum(unit, was)
                out[name][p, :, :kept] *= (was / unit)[:, None, None]
            out[name][p, :, kept:end] = part / unit[:, None, None]
            out[name + "_scales"][p] = unit


def attend64(s, new, held):
    case, (k, ks, v, vs), q = s["case"], s["cache"], s["q"].double()
    out, at = torch.zeros_like(q), 0
    for i, (n, h, tree) in enumerate(zip(new, held, trees(case, new))):
        if n and h:
            ids = s["pages"][i, :-(-h // case["page"])].long()
            hide = torch.zeros((n, h), dtype=torch.bool)
            for j, bits in enumerate(seen_by(tree)):
                for other in range(n):
                    hide[j, h - n + other] = not bits >> other & 1
            hide = hide.repeat_interleave(case["group"], 0).cuda()
            for head in range(case["heads"]):
                kd = k[ids, head].view(F8).double() * torch.exp2(ks[ids, head].double() - 127)[:, None, None]
                vd = v[ids, head].view(F8).double() * torch.exp2(vs[ids, head].double() - 127)[:, None, None]
                kd = kd.reshape(-1, case["dim"])[:h]
                vd = vd.transpose(1, 2).reshape(-1, case["dim"])[:h]
                of = slice(head * case["group"], (head + 1) * case["group"])
                z = torch.mm(q[at:at + n, of].reshape(-1, case["dim"]), kd.t().contiguous()) / math.sqrt(case["dim"])
                z.masked_fill_(hide, -math.inf)
                out[at:at + n, of] = torch.mm(torch.softmax(z, 1), vd).view(n, case["group"], case["dim"])
        at += n
    return out
