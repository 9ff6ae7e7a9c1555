"""MXFP4 in plain torch for the tests: the quantisation by its definition in 64 bits, and the
values of codes and scales.  On the CPU."""
import torch

GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def up(n, m):
    return -(-n // m) * m


def quantize(x, random=None):
    """[n, m] -> codes [n, 16 a block] uint8, scale codes [n, blocks] uint8 (64-bit arithmetic)."""
    n, m = x.shape
    kb = up(m, 32) // 32
    w = torch.zeros((n, kb * 32), dtype=torch.float64)
    w[:, :m] = x.double()
    w = w.view(n, kb, 32)
    bad = ~w.isfinite().all(2)
    w = torch.where(bad[:, :, None], 0.0, w)
    top = w.abs().amax(2)
    mant, e = torch.frexp(torch.where(top == 0, 1.0, top))  # top = mant 2^e, 1/2 <= mant < 1
    past = mant >= 0.875 if random is None else mant > 0.75
    code = (e - 1 - 2 + 127 + past.int()).clamp(min=0)
    # below 2^-125 the scale stays 2^-127: nothing lies past 6 there, and no step up is needed
    code = torch.where(e - 1 + 127 < 2, 0, code)
    code = torch.where(top == 0, 127, code)
    a = w.abs() * 2.0 ** (127 - code.double())[:, :, None]
    hi = torch.searchsorted(GRID, a.contiguous()).clamp(1, 7)
    share = (a - GRID[hi - 1]) / (GRID[hi] - GRID[hi - 1])
    if random is None:
        go = (share > 0.5) | ((share == 0.5) & (hi % 2 == 0))
    else:
        r = torch.zeros((n, kb * 32), dtype=torch.float64)
        r[:, :m] = random.double()
        go = share * 256 > r.view(n, kb, 32) + 0.5
    q = torch.where(go, hi, hi - 1) | torch.signbit(w).long() << 3
    q = torch.where(bad[:, :, None], 0, q).view(n, kb * 32).to(torch.uint8)
    return q[:, ::2] | q[:, 1::2] << 4, torch.where(bad, 255, code).to(torch.uint8)


def values(q, scale, cols):
    """Codes [n, >= 16 a block] and scale codes [n, >= blocks] -> [n, cols] in 64 bits."""
    kb = up(cols, 32) // 32
    q, scale = q[:, :16 * kb].cpu().long(), scale[:, :kb].cpu()
    c = torch.stack([q & 15, q >> 4], -1).flatten(1)
    v = torch.where(c >= 8, -GRID[c & 7], GRID[c & 7]).view(len(q), kb, 32)
    s = torch.where(scale == 255, float("nan"), 2.0 ** (scale.double() - 127))
    return (v * s[:, :, None]).flatten(1)[:, :cols]


def buffers(rows, cols, pad=0, fill=0, device="cpu"):
    """Codes and scales with the smallest strides and `pad` times 16 bytes more."""
    kb = up(cols, 32) // 32
    return (torch.full((rows, 16 * (kb + pad)), fill, dtype=torch.uint8, device=device),
            torch.full((rows, up(kb, 16) + 16 * pad), fill, dtype=torch.uint8, device=device))


def operand(x, pad=0, fill=0xff):
    """x quantised, in buffers whose pads hold `fill`."""
    q, s = buffers(x.shape[0], x.shape[1], pad, fill)
    a, b = quantize(x)
    q[:, :a.shape[1]], s[:, :b.shape[1]] = a, b
    return q, s
