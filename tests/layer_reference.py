"""Plain 64-bit forms of the transformer-layer operators, on the CPU, written
from their definitions in include/mx.h and independent of the package."""
import math

import torch

F8 = torch.float8_e4m3fn


def scale_byte(amax):
    """E8M0 byte of blocks with these largest magnitudes (float64 tensor)."""
    m, e = torch.frexp(amax)
    byte = (e.double() - 1 - 8 + 127).clamp(0, 254)
    byte = torch.where(amax > 0, byte, torch.zeros_like(byte))
    return torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255.0))


def pow2(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float64), byte.to(torch.int32) - 127)


def round_e4m3(u):
    """Nearest E4M3 value, ties to even, saturating at 448 (float64)."""
    _, e = torch.frexp(u.abs())
    step = torch.ldexp(torch.ones_like(u), (e - 1).clamp(min=-6) - 3)
    return (torch.round(u / step) * step).clamp(-448, 448)


def codes_of(u):
    """E4M3 values (float64, already rounded) as code bytes, -0 kept."""
    return u.to(torch.float32).to(F8).view(torch.uint8)


def spread(per_block, block, n):
    return per_block.repeat_interleave(block, -1)[..., :n]


def quantize(x, block):
    """x [rows, n] float64 -> codes uint8 [rows, n], bytes uint8 [rows, blocks]."""
    rows, n = x.shape
    nb = -(-n // block)
    xp = torch.nn.functional.pad(x, (0, nb * block - n)).view(rows, nb, block)
    amax = xp.abs().amax(2)
    amax = torch.where(torch.isnan(xp).any(2), torch.full_like(amax, math.nan), amax)
    byte = scale_byte(amax)
    bad = spread(byte, block, n) == 255
    u = torch.where(bad, torch.zeros_like(x), x) / pow2(spread(byte, block, n).clamp(max=254))
    code = codes_of(round_e4m3(u))
    sign = (torch.signbit(x).to(torch.uint8) << 7)
    return torch.where(bad, sign, code), byte.to(torch.uint8)


def dequantize(codes, byte, block):
    s = pow2(byte.double())
    s = torch.where(byte == 255, torch.full_like(s, math.nan), s)
    return codes.view(F8).double() * spread(s, block, codes.shape[-1])


def norm(x, weight, eps, residual=None):
    h = x.double() + (residual.double() if residual is not None else 0.0)
    s = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h, h * s * weight.double()


def norm_backward(dy, h, weight, eps, through=None):
    dy, h, w = dy.double(), h.double(), weight.double()
    k = h.shape[1]
    s = 1.0 / torch.sqrt(h.square().sum(1, keepdim=True) / k + eps)
    g = w * dy
    dx = s * (g - h * s * s * (g * h).sum(1, keepdim=True) / k)
    if through is not None:
        dx = dx + through.double()
    return dx, (dy * h * s).sum(0)


def append(cache, k, v, table, cu, lengths):
    """kv_append on CPU uint8 tensors, in place."""
    kc, ks, vc, vs = cache
    page = kc.shape[2]
    for i in range(table.shape[0]):
        a, n, held = int(cu[i]), int(cu[i + 1] - cu[i]), int(lengths[i])
        if n == 0:
            continue
        for j in range(held // page, -(-(held + n) // page)):
            if j >= table.shape[1]:
                break
            p = int(table[i, j])
            lo, hi = max(held, j * page), min(held + n, (j + 1) * page)
            kept, end = lo - j * page, hi - j * page
            for x, codes, scales, turn in ((k, kc, ks, False), (v, vc, vs, True)):
                new = x[a + lo - held:a + hi - held].double().transpose(0, 1)  # [head, token, dim]
                amax = new.abs().amax((1, 2))
                amax = torch.where(torch.isnan(new).any(2).any(1), torch.full_like(amax, math.nan), amax)
                was = scales[p].double()
                byte = scale_byte(amax)
                if kept:
                    byte = torch.maximum(byte, was)
                view = codes[p].transpose(1, 2) if turn else codes[p]            # [head, token, dim]
                for h in range(view.shape[0]):
                    if kept and byte[h] > was[h]:
                        old = view[h, :kept].clone()
                        if byte[h] == 255:
                            view[h, :kept] = old & 0x80
                        else:
                            u = old.view(F8).double() * 2.0 ** float(was[h] - byte[h])
                            view[h, :kept] = codes_of(round_e4m3(u))
                    if byte[h] == 255:
                        view[h, kept:end] = torch.signbit(new[h]).to(torch.uint8) << 7
                    else:
                        view[h, kept:end] = codes_of(round_e4m3(new[h] / pow2(byte[h])))
                scales[p] = byte.to(torch.uint8)


def attention(q, cache, table, cu, lengths, scale):
    """-> (out, bound): the exact result, and sum_j p_j |v_j| together with the
    largest sum_i |q_i k_i| * scale of a row, which the error bounds use."""
    kc, ks, vc, vs = cache
    page, heads = kc.shape[2], kc.shape[1]
    tokens, q_heads, dim = q.shape
    group = q_heads // heads
    out = torch.zeros((tokens, q_heads, dim), dtype=torch.float64)
    mag, reach = torch.zeros_like(out), torch.zeros((tokens, q_heads), dtype=torch.float64)

    def value(codes, byte):
        s = pow2(byte.double())
        s = torch.where(byte == 255, torch.full_like(s, math.nan), s)
        return codes.view(F8).double() * s[..., None, None]

    for i in range(table.shape[0]):
        a, n, length = int(cu[i]), int(cu[i + 1] - cu[i]), int(lengths[i])
        if n == 0 or length == 0:
            continue
        ids = table[i, :-(-length // page)].long()
        for h in range(heads):
            kd = value(kc[ids, h], ks[ids, h]).reshape(-1, dim)[:length]
            vd = value(vc[ids, h], vs[ids, h]).transpose(1, 2).reshape(-1, dim)[:length]
            for t in range(n):
                see = length - n + t + 1
                if see <= 0:
                    continue
                for g in range(group):
                    x = q[a + t, h * group + g].double()
                    z = kd[:see] @ x * scale
                    p = torch.softmax(z, 0)
                    out[a + t, h * group + g] = p @ vd[:see]
                    mag[a + t, h * group + g] = p @ vd[:see].abs()
                    reach[a + t, h * group + g] = (kd[:see].abs() @ x.abs()).max() * scale
    return out, mag, reach
