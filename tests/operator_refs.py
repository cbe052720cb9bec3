"""64-bit CPU statements of the gradient-making operators, for their tests,
and the rounding units their tolerances count.  Shares no code with the
library."""
import math

import torch

U32 = 2.0 ** -24                                             # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134}  # half the smallest subnormal


def f64(t):
    return t.detach().cpu().double()


def embedding(table, ids, scale):
    vocab = table.shape[0]
    ids = ids.cpu().reshape(-1).long()
    out = torch.zeros(ids.numel(), table.shape[1], dtype=torch.float64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < vocab:
            out[t] = f64(table[i]) * scale
    return out


def embedding_grad(dout, ids, vocab, scale):
    """(sum, sum of magnitudes, occurrences per row)"""
    ids = ids.cpu().reshape(-1).long()
    d = f64(dout).reshape(ids.numel(), dout.shape[-1])
    keep = (ids >= 0) & (ids < vocab)
    g = torch.zeros(vocab, d.shape[1], dtype=torch.float64)
    a = torch.zeros_like(g)
    g.index_add_(0, ids[keep], d[keep])
    a.index_add_(0, ids[keep], d[keep].abs())
    return g * scale, a * abs(scale), torch.bincount(ids[keep], minlength=vocab)


def layer_norm(x, gain, bias, eps):
    x = f64(x)
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + eps)
    y = xc * rstd[:, None] * f64(gain)
    return (y if bias is None else y + f64(bias)), mean, rstd


def layer_norm_grad(dy, x, gain, mean, rstd):
    """(dx, dgain, dbias, magnitudes of the terms of each)"""
    dy, r = f64(dy), f64(rstd)[:, None]
    xh = (f64(x) - f64(mean)[:, None]) * r
    gy = dy * f64(gain)
    c1, c2 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    dx = r * (gy - c1 - xh * c2)
    mag = r * (gy.abs() + gy.abs().mean(1, keepdim=True) + xh.abs() * (gy * xh).abs().mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), mag, (dy * xh).abs().sum(0), dy.abs().sum(0)


def e4m3_values():
    """The value of every code; 0x7f and 0xff are NaN."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if b & 0x7f == 0x7f:
            v = math.nan
        out.append(-v if b & 0x80 else v)
    return torch.tensor(out, dtype=torch.float64)


def checkpoint_values(codes, exponents, cols):
    v = e4m3_values()[codes.cpu().long()][:, :cols]
    e = exponents.cpu().long().repeat_interleave(128, 1)[:, :cols]
    f = torch.where(e == 255, torch.full((), math.nan, dtype=torch.float64), torch.pow(2.0, (e - 127).double()))
    return v * f


def checkpoint_encode(x):
    """(codes, exponents) by exhaustive search over the 127 magnitudes: the
    nearest, the even code on a tie."""
    x = f64(x)
    rows, cols = x.shape
    nb, pitch = (cols + 127) // 128, (cols + 15) // 16 * 16
    codes = torch.zeros(rows, pitch, dtype=torch.uint8)
    exps = torch.zeros(rows, nb, dtype=torch.uint8)
    mags = e4m3_values()[:127]
    for r in range(rows):
        for b in range(nb):
            blk = x[r, b * 128:(b + 1) * 128]
            big = blk.abs().max().item()
            if not math.isfinite(big):
                exps[r, b] = 255
                continue
            p = 0
            if big > 0:
                p = math.frexp(big)[1] - 9
                while 448.0 * 2.0 ** p < big:
                    p += 1
                while p > -124 and 448.0 * 2.0 ** (p - 1) >= big:
                    p -= 1
                p = max(p, -124)
            exps[r, b] = p + 127
            v = blk.abs() * 2.0 ** -p
            j = torch.searchsorted(mags, v).clamp(max=126)
            lo = (j - 1).clamp(min=0)
            dj, dl = (mags[j] - v).abs(), (v - mags[lo]).abs()
            best = torch.where((dl < dj) | ((dl == dj) & (lo % 2 == 0)), lo, j)
            sign = torch.signbit(blk).long() * 128
            codes[r, b * 128:b * 128 + blk.numel()] = (best + sign).to(torch.uint8)
    return codes, exps


def weight_grad(dy, values):
    d = f64(dy).reshape(values.shape[0], -1)
    return d.t() @ values, d.abs().t() @ values.abs()
