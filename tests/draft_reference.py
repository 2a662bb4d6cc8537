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
