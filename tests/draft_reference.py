"""Plain 64-bit forms of the operators of positions and drafted tokens, on the
CPU, written from their definitions in include/mx.h and independent of the
package."""
import torch


def table_of(length, rot, seed=0):
    """Cosines and sines of some angles, float32 (no two positions alike)."""
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(length, rot // 2, generator=g, dtype=torch.float64) * 6.283185307179586
    return torch.cat([a.cos(), a.sin()], 1).float()


def turn(x, table, positions, paired, back=False):
    """x [tokens, heads, dim] float64 rotated pair by pair; positions outside the
    table give NaN."""
    y, rot = x.clone(), table.shape[1]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if paired else (i, i + rot // 2)
        p = positions.long()
        inside = (p >= 0) & (p < table.shape[0])
        row = table[p.clamp(0, table.shape[0] - 1)].double()
        c = torch.where(inside, row[:, i], torch.nan)[:, None]
        s = torch.where(inside, row[:, rot // 2 + i], torch.nan)[:, None]
        if back:
            s = -s
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def heads(x, weight, eps, rotary):
    """Norm per head (weight None: none), then the rotation (table, positions, paired) or None."""
    y = x.double()
    if weight is not None:
        y = weight.double() * y / torch.sqrt(y.square().sum(2, keepdim=True) / y.shape[2] + eps)
    return turn(y, *rotary) if rotary is not None else y


def heads_backward(dy, x, weight, eps, rotary):
    """-> (dx, dweight, sum of |terms| of dweight); the last two None without a weight."""
    n = dy.double()
    if rotary is not None:
        n = turn(n, *rotary, back=True)
    if weight is None:
        return n, None, None
    x, w = x.double(), weight.double()
    s = 1.0 / torch.sqrt(x.square().sum(2, keepdim=True) / x.shape[2] + eps)
    g = w * n
    dx = s * (g - x * s * s * (g * x).sum(2, keepdim=True) / x.shape[2])
    terms = n * x * s
    return dx, terms.sum((0, 1)), terms.abs().sum((0, 1))


F8 = torch.float8_e4m3fn


def cache_value(codes, byte):
    s = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte.to(torch.int32) - 127)
    s = torch.where(byte == 255, torch.nan, s)
    return codes.view(F8).double() * s[..., None, None]


def ancestors(parents):
    """bool [n, n]: which nodes a node sees (itself and its ancestors)."""
    n = len(parents)
    sees = torch.zeros(n, n, dtype=torch.bool)
    for j, up in enumerate(parents):
        if up >= 0:
            sees[j] = sees[up]
        sees[j, j] = True
    return sees


def words_of(sees, words):
    """bool [n, m] -> int32 [n, words], bit b of a row being column b."""
    out = torch.zeros(sees.shape[0], words, dtype=torch.int64)
    for b in range(min(sees.shape[1], 32 * words)):
        out[:, b // 32] |= sees[:, b].long() << (b % 32)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).int()


def attention_tree(q, cache, table, cu, lengths, sees, scale):
    """sees[i]: bool [n, n] of sequence i's new tokens -> (out, sum_j p_j |v_j|, the
    largest sum |q_i k_i| * scale of a row)."""
    kc, ks, vc, vs = cache
    page, count = kc.shape[2], kc.shape[1]
    tokens, q_heads, dim = q.shape
    group = q_heads // count
    out = torch.zeros((tokens, q_heads, dim), dtype=torch.float64)
    mag, reach = torch.zeros_like(out), torch.zeros((tokens, q_heads), dtype=torch.float64)
    for i in range(table.shape[0]):
        a, n, length = int(cu[i]), int(cu[i + 1] - cu[i]), int(lengths[i])
        if n == 0 or length == 0:
            continue
        ids = table[i, :-(-length // page)].long()
        seen = torch.ones(n, length, dtype=torch.bool)
        for key in range(max(0, length - n), length):
            seen[:, key] = sees[i][:, key - (length - n)]
        for h in range(count):
            kd = cache_value(kc[ids, h], ks[ids, h]).reshape(-1, dim)[:length]
            vd = cache_value(vc[ids, h], vs[ids, h]).transpose(1, 2).reshape(-1, dim)[:length]
            for t in range(n):
                at = seen[t]
                if not bool(at.any()):
                    continue
                of = slice(h * group, (h + 1) * group)
                x = q[a + t, of].double()
                p = torch.softmax(x @ kd[at].t() * scale, 1)
                out[a + t, of] = p @ vd[at]
                mag[a + t, of] = p @ vd[at].abs()
                reach[a + t, of] = (x.abs() @ kd[at].abs().t()).amax(1) * scale
    return out, mag, reach


def verify(target, draft, ids, parents, cu, numbers, width):
    """-> (path, count, token) as lists, one sequence and node at a time."""
    def clean(p):
        p = p.double()
        return torch.where((p > 0) & torch.isfinite(p), p, 0.0)

    paths, counts, tokens = [], [], []
    vocab = target.shape[1]
    for i in range(len(cu) - 1):
        a, n = int(cu[i]), min(int(cu[i + 1] - cu[i]), 1024)
        path, token, node = [], -1, 0
        while n > 0:
            path.append(node)
            row = a + node
            kids = [j for j in range(node + 1, n) if int(parents[a + j]) == node]
            if len(path) >= width:
                kids = []
            p = clean(target[row])
            w = p
            if draft is not None and kids:
                x, q = int(ids[a + kids[0]]), clean(draft[row])
                if 0 <= x < vocab and float(numbers[row, 0]) * float(q[x]) < float(p[x]):
                    node = kids[0]
                    continue
                kids = kids[1:]
                w = (p - q).clamp(min=0)
                if float(w.sum()) <= 0:
                    w = p
            token = -1
            total = float(w.sum())
            if total > 0:
                past = (w.cumsum(0) > float(numbers[row, 1]) * total) & (w > 0)
                at = torch.nonzero(past if bool(past.any()) else w > 0)
                token = int(at[0]) if bool(past.any()) else int(at[-1])
            follow = [j for j in kids if int(ids[a + j]) == token and token >= 0]
            if not follow:
                break
            node = follow[0]
        paths.append(path + [-1] * (width - len(path)))
        counts.append(len(path))
        tokens.append(token)
    return paths, counts, tokens


def keep(cache, table, lengths, path, count):
    """kv_keep on CPU uint8 tensors, in place."""
    kc, ks, vc, vs = cache
    pool, page = kc.shape[0], kc.shape[2]

    def moved(codes, by, to):
        """[.., dim] codes at byte `by` as codes at byte `to`."""
        if to == by:
            return codes.clone()
        if to == 255:
            return codes & 0x80
        u = codes.view(F8).double() * 2.0 ** (int(by) - int(to))
        _, e = torch.frexp(u.abs())
        step = torch.ldexp(torch.ones_like(u), (e - 1).clamp(min=-6) - 3)
        return (torch.round(u / step) * step).float().to(F8).view(torch.uint8)

    for i in range(table.shape[0]):
        held, nodes = int(lengths[i]), []
        for j in range(min(int(count[i]), path.shape[1])):
            p = int(path[i, j])
            if p <= (nodes[-1] if nodes else -1) or (held + p) // page >= table.shape[1]:
                break
            nodes.append(p)
        first = 0
        while first < len(nodes) and nodes[first] == first:
            first += 1
        if held < 0 or first == len(nodes):
            continue
        for codes, scales, turn in ((kc, ks, False), (vc, vs, True)):
            for h in range(codes.shape[1]):
                def rows(p):
                    return codes[p, h].t() if turn else codes[p, h]
                came = []
                for p in nodes:
                    at = int(table[i, (held + p) // page])
                    if 0 <= at < pool:
                        came.append((rows(at)[(held + p) % page].clone(), int(scales[at, h])))
                    else:
                        came.append((torch.zeros(rows(0).shape[1], dtype=torch.uint8), 0))
                for pg in range((held + first) // page, (held + len(nodes) - 1) // page + 1):
                    lo, hi = max(held + first, pg * page), min(held + len(nodes), (pg + 1) * page)
                    at, kept = int(table[i, pg]), lo - pg * page
                    if not 0 <= at < pool:
                        continue
                    was = int(scales[at, h]) if kept else 0
                    byte = max([was] + [came[p - held][1] for p in range(lo, hi)])
                    view = rows(at)
                    if kept and byte > was:
                        view[:kept] = moved(view[:kept].contiguous(), was, byte)
                    for p in range(lo, hi):
                        view[p - pg * page] = moved(came[p - held][0], came[p - held][1], byte)
                    scales[at, h] = byte
