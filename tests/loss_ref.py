"""Plain 64-bit definitions of the losses behind the output layer, and the
error bounds their results are held to.

Every function gives (value, bound) pairs in 64 bits.  The bounds count these
roundings (e = 2^-24, the unit roundoff of fp32; u of the 16-bit type):

  - an exponential 2^(x k - c): k = log2(e) / T is rounded once and the fused
    multiply-add once, each e times the exponent y log2(e) with y the distance
    to the largest logit over T, so 2 |y| e of the value; the hardware's 2^x is
    within 2^-22 = 4 e: (2 |y| + 4) e together;
  - a sum of n exponentials: a lane adds at most n / 128 + 136 of them one after another (rows
    of up to 4,096 have 32 lanes, others 128 at least), e each; a dozen partial sums at most
    are joined on any way from a lane to the result, each with an exponential and two
    roundings (6 e); the exponentials' own errors average to at most (2 log n + 4) e, log n <=
    13: below (n / 128 + 136 + 72 + 30) e, for which (n / 128 + 300) e stands;
  - lse = c ln 2 + log s: the sum's relative error, k's rounding (e |m / T|) and
    four roundings of the parts;
  - lp below -log 2: the sum's error and 2^-21 of the parts; above it lp =
    -log1p(R / e), whose relative error is that of R / e;
  - 1 - p = R / (R + e): relative errors of both;
  - an exponential below 2^-126, the least normal number, is zero: a sum relative to
    its largest term, so of at least 1, or R relative to such a sum, loses less than
    n 2^-126 to them, and 2^-125 n with the rounding of what is just above;
  - one rounding to 16 bits, u of the value or half the type's smallest subnormal:
    2^-25 of binary16, 2^-134 of bfloat16.
"""
from __future__ import annotations

import math

import torch

from train_ref import E32, U

LN2 = math.log(2.0)
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def sum_error(n):
    return (n / 128 + 300) * E32


def rounded(value, bound, dtype):
    """The bound of a result that is rounded once to 16 bits, of a value that is
    off by `bound` before: the value may move the rounding, by u of it."""
    return bound + U[dtype] * (value.abs() + bound) + TINY[dtype]


class Rows:
    """Softmax statistics of rows of logits at temperature T."""

    def __init__(self, logits, targets, temp, there):
        x = logits.double() / temp
        self.x, self.there = x, there
        n = x.shape[1]
        self.n = n
        self.m = x.amax(1)
        self.lse = torch.logsumexp(x, 1)
        self.y = (x - self.m[:, None]).abs()
        self.logp_all = x - self.lse[:, None]
        self.p = self.logp_all.exp()
        row = torch.arange(x.shape[0], device=x.device)
        self.row, self.t = row, targets.clamp(min=0)
        self.lp = self.logp_all[row, self.t]
        # exact 1 - p of the target, from the others
        rest = x.clone()
        rest[row, self.t] = -math.inf
        self.rest = (torch.logsumexp(rest, 1) - self.lse).exp()
        self.lp = torch.where(self.rest < 0.5, torch.log1p(-self.rest), self.lp)
        es = sum_error(n)
        yt = self.y[row, self.t]
        finite = torch.isfinite(self.lp)
        lost = n * 2.0 ** -125
        near = self.lp.abs() * (2 * es + (2 * yt + 20) * E32) + lost
        far = es + 8 * E32 * (self.lp.abs() + math.log(n) + yt + 1)
        self.lp_tol = torch.where(finite, torch.where(self.lp > -LN2, near, far), torch.zeros_like(far))
        # the two branches meet at -log 2, where either may have been taken
        self.lp_tol = torch.where((self.lp + LN2).abs() < 1e-3, torch.maximum(near, far), self.lp_tol)
        self.lse_tol = es + 4 * E32 * (self.m.abs() + self.lse.abs() + math.log(n) + 1)
        self.p_tol = self.p * (es + (2 * torch.where(self.p > 0, self.y, torch.zeros_like(self.y)) + 20) * E32) + 2.0 ** -126
        self.rest_tol = self.rest * (2 * es + 20 * E32 + 2 * yt.clamp(max=200) * E32) + lost

    def masked(self, v):
        keep = self.there.reshape([-1] + [1] * (v.dim() - 1))
        return torch.where(keep, v, torch.zeros_like(v))

    def slope_grad(self, slope, slope_tol, dtype):
        """slope * (one at the target - p), and its bound."""
        g = -slope[:, None] * self.p
        tol = slope.abs()[:, None] * self.p_tol + slope_tol[:, None] * self.p + 4 * E32 * g.abs()
        g[self.row, self.t] = slope * self.rest
        tol[self.row, self.t] = slope.abs() * self.rest_tol + slope_tol * self.rest + 4 * E32 * (slope * self.rest).abs()
        return self.masked(g), rounded(self.masked(g), self.masked(tol), dtype)


def logprob(logits, targets, temp):
    r = Rows(logits, targets, temp, (targets >= 0) & (targets < logits.shape[1]))
    return r


def logprob_backward(logits, targets, temp, d_logp, dtype):
    r = logprob(logits, targets.clamp(max=logits.shape[1] - 1), temp)
    r.there = (targets >= 0) & (targets < logits.shape[1])
    s = d_logp.double() / temp
    return r.slope_grad(s, 2 * E32 * s.abs(), dtype)


def distill(logits, top, top_ids, temp, soft, targets, hard, weight, scale, dtype):
    """((loss, bound), (d_logits, bound))"""
    t, v = logits.shape
    dev = logits.device
    there = torch.ones(t, dtype=torch.bool, device=dev)
    y = torch.zeros(t, dtype=torch.int64, device=dev)
    if targets is not None:
        there, y = (targets >= 0) & (targets < v), targets.clamp(0, v - 1).long()
    w = weight.double() if weight is not None else torch.ones(t, dtype=torch.float64, device=dev)
    loss = torch.zeros(t, dtype=torch.float64, device=dev)
    loss_tol = torch.zeros_like(loss)
    grad = torch.zeros(t, v, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(grad)
    if top is not None and top.shape[1]:
        r = Rows(logits, y, temp, there)
        k = top.shape[1]
        ids = top_ids.reshape(t, k).long()
        here = (ids >= 0) & (ids < v) & (top != -math.inf)
        ids = ids.clamp(0, v - 1)
        z = torch.where(here, top.double() / temp, torch.full((), -math.inf, dtype=torch.float64, device=dev))
        some = here.any(1)
        lse = torch.where(some, torch.logsumexp(z, 1), torch.zeros_like(w))
        q = torch.where(here, (z - lse[:, None]).exp(), torch.zeros_like(z))
        q_tol = q * (k * E32 + (2 * (z - lse[:, None]).nan_to_num(0, 0, 0).abs() + 150) * E32)
        a = torch.where(some, soft * temp * torch.ones_like(w), torch.zeros_like(w))
        diff = torch.where(q > 0, (z - lse[:, None]) - r.logp_all.gather(1, ids), torch.zeros_like(z))
        part = torch.where(some, soft * temp ** 2 * (q * diff).sum(1), torch.zeros_like(w))
        mag = torch.where(q > 0, q * (z - r.x.gather(1, ids)).abs(), torch.zeros_like(z)).sum(1)
        loss = loss + part
        # sum q (t - x) / T and the two sums' logarithms, each with its own error
        loss_tol = loss_tol + abs(soft) * temp ** 2 * torch.where(
            some, (q_tol * diff.abs()).sum(1) + mag * (k + 40) * E32 + sum_error(v) + (k + 150) * E32
            + 16 * E32 * (r.lse.abs() + lse.abs() + math.log(v) + 10 + mag), torch.zeros_like(w))
        dense, dense_tol = torch.zeros_like(grad), torch.zeros_like(grad)
        dense.scatter_add_(1, ids, q)
        dense_tol.scatter_add_(1, ids, q_tol + 4 * E32 * q)
        grad += a[:, None] * (r.p - dense)
        tol += a.abs()[:, None] * (r.p_tol + dense_tol + 8 * E32 * (r.p + dense))
    if hard:
        r = Rows(logits, y, 1.0, there)
        loss = loss - hard * r.lp
        loss_tol = loss_tol + abs(hard) * (r.lp_tol + 4 * E32 * r.lp.abs())
        p, p_tol = r.p.clone(), r.p_tol.clone()
        p[r.row, r.t], p_tol[r.row, r.t] = -r.rest, r.rest_tol
        grad += hard * p
        tol += abs(hard) * (p_tol + 8 * E32 * p.abs())
    loss, loss_tol = w * loss, w.abs() * (loss_tol + 8 * E32 * loss.abs())
    grad, tol = grad * (w * scale)[:, None], tol * (w * scale).abs()[:, None]
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    pick = lambda x: torch.where(there.reshape([-1] + [1] * (x.dim() - 1)), x, zero)   # noqa: E731
    return (pick(loss), pick(loss_tol)), (pick(grad), rounded(pick(grad), pick(tol), dtype))


def policy(logits, targets, temp, old, ref, adv, weight, low, high, kl, scale, dtype):
    """((loss, bound), (logp, bound), (d_logits, bound))"""
    v = logits.shape[1]
    there = (targets >= 0) & (targets < v)
    r = Rows(logits, targets.clamp(0, v - 1), temp, there)
    a, w = adv.double(), weight.double() if weight is not None else torch.ones_like(r.lp)
    move = r.lp - old.double()
    ratio = move.exp()
    ratio_tol = ratio * (r.lp_tol + 2 * E32 * (move.abs() + r.lp.abs()) + 8 * E32)
    lo, hi = 1.0 - low, 1.0 + high
    limit = torch.where(a > 0, hi * a, lo * a)
    inside = ratio * a <= torch.where(a >= 0, ratio.clamp(lo, hi) * a, ratio.clamp(lo, hi) * a)
    loss = torch.where(inside, -ratio * a, -limit)
    slope = torch.where(inside, -ratio * a, torch.zeros_like(a))
    loss_tol = a.abs() * torch.where(inside, ratio_tol + 4 * E32 * ratio, torch.full_like(a, 4 * E32 * (hi + 1)))
    slope_tol = torch.where(inside, a.abs() * (ratio_tol + 4 * E32 * ratio), torch.zeros_like(a))
    if kl:
        d = ref.double() - r.lp
        d_tol = r.lp_tol + 2 * E32 * (d.abs() + r.lp.abs())
        loss = loss + kl * (torch.expm1(d) - d)
        loss_tol = loss_tol + abs(kl) * (torch.expm1(d).abs() * d_tol + d_tol ** 2 * d.exp()
                                         + 16 * E32 * (torch.expm1(d) - d).abs())
        slope = slope - kl * torch.expm1(d)
        slope_tol = slope_tol + abs(kl) * (d.exp() * d_tol + 8 * E32 * torch.expm1(d).abs())
    loss, slope = w * loss, w * slope * scale / temp
    loss_tol = w.abs() * loss_tol + 4 * E32 * loss.abs()
    slope_tol = (w * scale / temp).abs() * slope_tol + 8 * E32 * slope.abs()
    return ((r.masked(loss), r.masked(loss_tol)), (r.masked(r.lp), r.masked(r.lp_tol)),
            r.slope_grad(slope, slope_tol, dtype))


def preference(logits, targets, starts, ref, beta, smoothing, scale, dtype):
    """((loss, bound), (reward, bound), (logp, bound), (d_logits, bound))"""
    t, v = logits.shape
    at = starts.tolist()
    rows = torch.arange(t, device=logits.device)
    there = (targets >= 0) & (targets < v) & (rows >= at[0]) & (rows < at[-1])
    r = Rows(logits, targets.clamp(0, v - 1), 1.0, there)
    gain = r.masked(r.lp - ref.double() if ref is not None else r.lp)
    tol = r.masked(r.lp_tol)
    s = torch.stack([gain[a:b].sum() for a, b in zip(at, at[1:])])
    s_tol = torch.stack([tol[a:b].sum() for a, b in zip(at, at[1:])])
    reward, reward_tol = beta * s, abs(beta) * s_tol
    m = reward[0::2] - reward[1::2]
    m_tol = reward_tol[0::2] + reward_tol[1::2] + E32 * m.abs()
    ls = torch.nn.functional.logsigmoid
    loss = -(1 - smoothing) * ls(m) - smoothing * ls(-m)
    loss_tol = m_tol + 16 * E32 * (loss.abs() + m.abs() * smoothing)
    down, up = torch.sigmoid(-m), torch.sigmoid(m)
    dm = (smoothing * up - (1 - smoothing) * down) * beta
    dm_tol = abs(beta) * (up * down * m_tol + 16 * E32 * (smoothing * up + (1 - smoothing) * down))
    slope, slope_tol = torch.zeros_like(r.lp), torch.zeros_like(r.lp)
    for i, (a, b) in enumerate(zip(at, at[1:])):
        slope[a:b] = (dm[i // 2] if i % 2 == 0 else -dm[i // 2]) * scale
        slope_tol[a:b] = dm_tol[i // 2] * abs(scale)
    return ((loss, loss_tol), (reward, reward_tol + 2 * E32 * reward.abs()), (r.masked(r.lp), r.masked(r.lp_tol)),
            r.slope_grad(slope, slope_tol + 2 * E32 * slope.abs(), dtype))
