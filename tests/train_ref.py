"""Plain 64-bit definitions of the training operators, and the error bounds
their 16-bit results are held to.

u(dtype) is the unit roundoff of a 16-bit type (2^-11 binary16, 2^-8
bfloat16): one rounding of a value r moves it by at most u |r| (plus 2^-25 for
a binary16 subnormal).  A sum of n fp32 terms, in any order, is within
n 2^-24 sum |terms| of the exact one (first order); each product or other fp32
operation adds 2^-24 of its result.
"""
from __future__ import annotations

import torch

BLOCK = 32
LIMITS = {"f16": (-24, 9), "bf16": (-127, 121)}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
E32 = 2.0 ** -24


def two_to(k):
    """2^k, exact, for whole k (64 bits)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def pack(x, dtype):
    """(q int8 [rows, cols], s uint8 [rows, blocks]) of the values x."""
    x = x.double().cpu()
    rows, cols = x.shape
    lo, hi = LIMITS[dtype]
    nb = -(-cols // BLOCK)
    q = torch.zeros(rows, nb * BLOCK, dtype=torch.int8)
    s = torch.zeros(rows, nb, dtype=torch.uint8)
    for b in range(nb):
        blk = x[:, b * BLOCK:(b + 1) * BLOCK]
        bad = ~torch.isfinite(blk).all(1)
        a = torch.where(bad, torch.zeros(rows, dtype=torch.float64),
                        blk.abs().nan_to_num(0.0, 0.0, 0.0).amax(1))
        k = torch.full((rows,), lo)
        for kk in range(hi - 1, lo - 1, -1):   # the smallest k with a <= 127 * 2^k
            k = torch.where((k == lo) & (a > 127.0 * 2.0 ** kk), torch.full_like(k, kk + 1), k)
        v = (blk / two_to(k)[:, None]).round().clamp(-127, 127)
        q[:, b * BLOCK:b * BLOCK + blk.shape[1]] = \
            torch.where(bad[:, None], torch.zeros_like(v), v).to(torch.int8)
        s[:, b] = torch.where(bad, torch.full_like(k, 255), k + 127).to(torch.uint8)
    return q[:, :cols], s


def values(q, s):
    """What a checkpoint stands for (64 bits)."""
    step = two_to(s.long() - 127)
    step = torch.where(s == 255, torch.full_like(step, float("nan")), step)
    cols = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * step[:, cols]


def norm_forward(x, res, gain, eps):
    """(h, rstd, xhat, y)."""
    h = x.double() + (res.double() if res is not None else 0.0)
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    xhat = h * rstd[:, None]
    return h, rstd, xhat, xhat * gain.double() if gain is not None else xhat


def norm_backward(dy, xhat, rstd, gain, dres):
    """(dx, d_gain, bound on dx's fp32 error, sum of |terms| of d_gain)."""
    dy, rstd = dy.double(), rstd.double()[:, None]
    u = dy * gain.double() if gain is not None else dy
    n = dy.shape[1]
    mean = (u * xhat).sum(1, keepdim=True) / n
    size = (u * xhat).abs().sum(1, keepdim=True) / n
    dx = rstd * (u - xhat * mean)
    # u and its products: 3 roundings a term, a sum of n terms, then 5 more operations
    err = rstd * (xhat.abs() * size * (n + 8) * E32 + (u.abs() + xhat.abs() * size) * 8 * E32)
    if dres is not None:
        dx = dx + dres.double()
        err = err + (dres.double().abs() + dx.abs()) * 2 * E32
    return dx, (dy * xhat).sum(0), err, (dy * xhat).abs().sum(0)


def embed_grad(d_out, ids, scale, vocab, old=None):
    """(d_table, sum of |terms|, count of terms) of every table row."""
    ids = ids.flatten().long().to(d_out.device)
    keep = (ids >= 0) & (ids < vocab)
    total = torch.zeros(vocab, d_out.shape[1], dtype=torch.float64, device=d_out.device)
    size, count = total.clone(), torch.zeros(vocab, dtype=torch.float64, device=d_out.device)
    total.index_add_(0, ids[keep], d_out[keep].double())
    size.index_add_(0, ids[keep], d_out[keep].double().abs())
    count.index_add_(0, ids[keep], torch.ones_like(ids[keep], dtype=torch.float64))
    total, size = total * scale, size * abs(scale)
    if old is not None:
        total, size = total + old.double(), size + old.double().abs()
    return total, size, count


def weight_grad(dy, x, gain, old=None):
    """(dw, sum of |terms|) with x in 64 bits."""
    dw, size = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
    if gain is not None:
        dw, size = dw * gain.double(), size * gain.double().abs()
    if old is not None:
        dw, size = dw + old.double(), size + old.double().abs()
    return dw, size


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound, element by element; NaN where ref has NaN."""
    got, ref = got.double(), ref.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    off = ((got - ref).abs() - bound)[~nan]
    assert off.numel() == 0 or float(off.max()) <= 0.0, \
        f"{what}: {int((off > 0).sum())} of {off.numel()} beyond the bound, by up to {float(off.max()):.3g}"
