"""The losses behind the output layer on the GPU against their definitions in 64
bits, at the sizes, strides, masks and values where they can go wrong.  The
bounds are those of the roundings that the operators document (loss_ref)."""
import math

import pytest
import torch

import loss_ref as ref
import loss_rule as rule
import zero_sharded_optimizer_02_gb300 as z
from train_ref import TYPES

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = ["f16", "bf16"]
# one element, below and above a vector, around a warp's and a CTA's share, wide, the widest
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (33, 63), (3, 1000), (7, 4097), (700, 257), (130, 2048),
         (1, 50257), (9, 50257), (2, 131072), (3, 131079), (1, 393216), (2, 393211)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Banded:
    """A matrix inside a larger buffer whose other elements must stay as they are."""

    def __init__(self, rows, cols, dtype, fill=None, extra=16):
        self.pitch = -(-cols // 8) * 8 + extra
        self.buf = torch.full((64 + rows * self.pitch + 64,), 77, dtype=dtype, device=DEV)
        self.t = self.buf[64:64 + rows * self.pitch].view(rows, self.pitch)[:, :cols]
        if fill is not None:
            self.t.copy_(fill)
        self.before = self.buf.clone()

    def check(self, what="matrix"):
        inside = torch.zeros_like(self.buf, dtype=torch.bool)
        torch.as_strided(inside, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(True)
        assert torch.equal(self.buf[~inside], self.before[~inside]), f"{what}: written outside its elements"


class Vec(Banded):
    """A vector of n fp32 elements between others that must stay as they are."""

    def __init__(self, n):
        super().__init__(1, n, torch.float32, extra=8)
        self.v = self.t[0]


def space(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)


def near(got, want, what):
    value, bound = want
    assert got.shape == value.shape, what
    off = (got.double() - value).abs() - bound
    assert not bool((~(off <= 0)).any()), \
        f"{what}: {int((~(off <= 0)).sum())} of {off.numel()} beyond the bound, worst by {float(off.max())}"


def batch(seed, rows, vocab, dtype, pad=0.2, sigma=2.0, masked=0):
    """Logits, with the first `masked` columns at -inf, and targets, some of them padding; what is padded holds NaN."""
    g = gen(seed)
    x = sigma * torch.randn(rows, vocab, generator=g, device=DEV)
    x[:, :masked] = -math.inf
    targets = torch.randint(masked, vocab, (rows,), generator=g, device=DEV)
    boost = sigma * 9 * torch.rand(rows, generator=g, device=DEV)
    x[torch.arange(rows, device=DEV), targets] += boost.clamp(max=3e4)
    gone = torch.rand(rows, generator=g, device=DEV) < pad
    targets[gone] = -1 - torch.randint(0, 200, (rows,), generator=g, device=DEV)[gone]
    x[gone] = math.nan
    return g, Banded(rows, vocab, TYPES[dtype], x).t, targets


def vec(g, rows, sigma=1.0, gone=None):
    v = sigma * torch.randn(rows, generator=g, device=DEV)
    if gone is not None:
        v[gone] = math.nan
    return v


def grad_of(logits):
    return Banded(logits.shape[0], logits.shape[1], logits.dtype, extra=24)


# -- log-probabilities ------------------------------------------------------------


def check_logprob(x, targets, temp, ids=None):
    t, n = x.shape
    lp, lse = Vec(t), Vec(t)
    z.zero_token_logprob(z.mat(x), z.ids(ids if ids is not None else targets), temp, lp.v, lse.v)
    r = ref.logprob(x, targets.clamp(max=n - 1), temp)
    r.there = (targets >= 0) & (targets < n)
    near(lp.v, (r.masked(r.lp), r.masked(r.lp_tol)), "logp")
    near(lse.v, (r.masked(r.lse), r.masked(r.lse_tol)), "lse")
    lp.check()
    lse.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_logprob(dtype, rows, vocab):
    _, x, targets = batch(rows + vocab, rows, vocab, dtype)
    check_logprob(x, targets, 1.0)
    check_logprob(x, targets, 0.6, targets.int())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sigma,temp", [(0.0, 1.0), (50.0, 1.0), (1000.0, 1.0), (1000.0, 300.0), (3.0, 2.0 ** -20), (3.0, 2.0 ** 20)])
def test_logprob_spreads(dtype, sigma, temp):
    _, x, targets = batch(3, 17, 1111, dtype, sigma=sigma)
    check_logprob(x, targets, temp)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logprob_far_from_zero(dtype):
    """Rows whose logits are all large, where only differences count."""
    x = torch.full((4, 100), 60000.0, device=DEV)
    x[1], x[2] = -60000.0, 0.0
    x[3] = torch.linspace(-60000.0, 60000.0, 100, device=DEV)
    x = x.to(TYPES[dtype])
    x = Banded(4, 100, x.dtype, x).t
    check_logprob(x, torch.tensor([5, 6, 7, 99], device=DEV), 1.0)


def test_one_output_of_two():
    _, x, targets = batch(11, 40, 333, "bf16")
    a, b = Vec(40), Vec(40)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, a.v, b.v)
    c, d = Vec(40), Vec(40)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, c.v, None)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, None, d.v)
    assert torch.equal(a.v, c.v) and torch.equal(b.v, d.v)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_logprob_backward(dtype, rows, vocab):
    g, x, targets = batch(2 * rows + vocab, rows, vocab, dtype)
    d_lp = vec(g, rows, 3.0, targets < 0)
    for temp in (1.0, 1.7):
        d = grad_of(x)
        z.zero_token_logprob_backward(z.mat(x), z.ids(targets), temp, d_lp, z.mat(d.t))
        near(d.t, ref.logprob_backward(x, targets, temp, torch.where(targets < 0, 0.0, d_lp), dtype), "d_logits")
        d.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(3, 1000), (40, 50257), (700, 2049), (2, 131072)])
def test_gradient_in_the_place_of_the_logits(dtype, rows, vocab):
    g, x, targets = batch(5, rows, vocab, dtype)
    d_lp = vec(g, rows)
    d = grad_of(x)
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, d_lp, z.mat(d.t))
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, d_lp, z.mat(x))
    assert torch.equal(x, d.t)


def test_gradient_against_differences():
    """The loss's own differences, in a vocabulary small enough to move every logit."""
    g, x, targets = batch(9, 6, 12, "f16", pad=0.0)
    x.mul_(0.25)
    d_lp = vec(g, 6)
    d = grad_of(x)
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, d_lp, z.mat(d.t))
    step = 2.0 ** -5
    up, down = Vec(6), Vec(6)
    for j in range(12):
        hi, lo = x.clone(), x.clone()
        hi[:, j] += step
        lo[:, j] -= step
        width = (hi[:, j].double() - lo[:, j].double())
        hi, lo = Banded(6, 12, x.dtype, hi).t, Banded(6, 12, x.dtype, lo).t
        z.zero_token_logprob(z.mat(hi), z.ids(targets), 1.0, up.v)
        z.zero_token_logprob(z.mat(lo), z.ids(targets), 1.0, down.v)
        slope = d_lp.double() * (up.v.double() - down.v.double()) / width
        # the third derivative of log softmax is below 1/8, so a central difference is off by less than
        # step^2 / 48 (times 2 for the uneven steps that rounding leaves); logp itself by 2^-16 at this size
        bound = d_lp.double().abs() * (step ** 2 / 24 + 2.0 ** -16 / step + width * 0) + 2.0 ** -11 * d.t[:, j].double().abs() + 2.0 ** -10 * d_lp.double().abs()
        assert bool(((d.t[:, j].double() - slope).abs() <= bound).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks_and_special_rows(dtype):
    """-inf is an entry that cannot be chosen; a NaN, +inf or nothing but -inf gives NaN."""
    n = 2500
    g, x, _ = batch(21, 8, n, dtype, pad=0.0)
    targets = torch.tensor([5, 7, 0, 0, 1, 2, 3, n - 1], device=DEV)
    inf = math.inf
    x[0, ::2] = -inf                      # target 5 stays
    x[1, 1::2] = -inf                     # target 7 is among the masked
    x[2, 1:] = -inf                       # only the target is left
    x[3] = -inf                           # nothing is left
    x[4, 2000] = math.nan
    x[5, 2] = math.nan                    # the target itself
    x[6, 100] = inf
    x[7, n - 1] = inf                     # the target itself
    lp, lse = Vec(8), Vec(8)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, lp.v, lse.v)
    r = ref.Rows(x[:3], targets[:3], 1.0, torch.ones(3, dtype=torch.bool, device=DEV))
    near(lse.v[:3], (r.lse, r.lse_tol), "lse")
    near(lp.v[:1], (r.lp[:1], r.lp_tol[:1]), "logp")
    assert float(lp.v[1]) == -inf and float(lp.v[2]) == 0.0
    assert bool(torch.isnan(lp.v[3:]).all())
    d = grad_of(x)
    one = torch.ones(8, device=DEV)
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, one, z.mat(d.t))
    assert bool((d.t[0, ::2] == 0).all())
    assert float(d.t[1, 7]) == 1.0 and bool((d.t[1, 9::2] == 0).all())
    assert bool((d.t[2] == 0).all())
    assert bool(torch.isnan(d.t[3:].float()).any(1).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [60, 5000])
def test_masks_of_a_low_value(dtype, vocab):
    """Masks of the type's lowest value and of others that no logit comes near.  Rows that they leave nothing of: uniform
    within 2^30 log 2 = 7.4e8 of zero, NaN beyond, where they count as -inf."""
    low = torch.finfo(TYPES[dtype]).min
    g, x, targets = batch(23, 12, vocab, dtype, pad=0.0)
    targets[:] = torch.arange(12, device=DEV)
    x[0, 12:] = low
    x[1, ::2] = low
    x[2, 12:] = -30000.0
    x[3, :] = -30000.0
    x[4, :] = 60000.0
    x[5, :] = low
    x[5, 5] = 1.0
    x[6, 20:] = max(-1e10, low)
    x[7, 20:] = max(-1e20, low)
    x[8, 20:] = max(-2e9, low)
    x[9, :] = max(-5e8, low)
    x[10, :] = max(-1e12, low)
    x[11, :] = low
    gone = [10, 11] if dtype == "bf16" else []
    kept = [i for i in range(12) if i not in gone]
    y = Banded(len(kept), vocab, x.dtype, x[kept]).t
    t = targets[kept].contiguous()
    check_logprob(y, t, 1.0)
    one = torch.ones(len(kept), device=DEV)
    d = grad_of(y)
    z.zero_token_logprob_backward(z.mat(y), z.ids(t), 1.0, one, z.mat(d.t))
    near(d.t, ref.logprob_backward(y, t, 1.0, one, dtype), "d_logits")
    # a teacher's entries on masked logits: an infinite loss where those count as -inf, so not of these rows
    near_ones = [i for i in range(12) if bool((x[i].double().abs() < 7e8).all())]
    y = Banded(len(near_ones), vocab, x.dtype, x[near_ones]).t
    top, ids = teacher(g, y, 5)
    check_distill(y, top, ids, 2.0, 0.5, targets[near_ones].contiguous(), 0.5, None, 1.0, dtype)
    if gone:
        lp, d = torch.empty(12, device=DEV), grad_of(x)
        z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, lp)
        z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, torch.ones(12, device=DEV), z.mat(d.t))
        assert bool(torch.isnan(lp[gone]).all()) and bool(torch.isfinite(lp[kept]).all())
        assert bool(torch.isnan(d.t[gone].float()).any(1).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_far_from_zero(dtype):
    """Rows whose logits are all large, where only differences count."""
    g = gen(29)
    x = torch.randn(6, 700, generator=g, device=DEV) * 300
    x += torch.tensor([60000.0, -60000.0, 20000.0, -3000.0, 1000.0, 0.0], device=DEV)[:, None]
    x = Banded(6, 700, TYPES[dtype], x).t
    t = torch.arange(6, device=DEV)
    one = torch.ones(6, device=DEV)
    for temp in (1.0, 100.0):
        check_logprob(x, t, temp)
        d = grad_of(x)
        z.zero_token_logprob_backward(z.mat(x), z.ids(t), temp, one, z.mat(d.t))
        near(d.t, ref.logprob_backward(x, t, temp, one, dtype), "d_logits")


def test_targets_beyond_the_vocabulary():
    g, x, targets = batch(4, 50, 300, "bf16", pad=0.0)
    targets[::7] = 300
    targets[3] = 1 << 40
    want = torch.where(targets < 300, targets, torch.full_like(targets, -1))
    for fn in ("logprob", "backward"):
        out = []
        for t, flagged in ((targets, 1), (want, 0)):
            bad = torch.zeros(1, dtype=torch.int32, device=DEV)
            if fn == "logprob":
                o = torch.empty(50, device=DEV)
                z.zero_token_logprob(z.mat(x), z.ids(t), 1.0, o, None, bad)
            else:
                o = grad_of(x).t
                z.zero_token_logprob_backward(z.mat(x), z.ids(t), 1.0, torch.ones(50, device=DEV), z.mat(o), bad)
            assert int(bad) == flagged
            out.append(o)
        assert torch.equal(*out)


# -- distillation and cross-entropy -------------------------------------------------


def teacher(g, x, k, gaps=True, repeat=True):
    """Teacher entries: any numbers, some absent, some twice, some rows without any."""
    rows, n = x.shape
    top = Banded(rows, k, x.dtype, 2.0 * torch.randn(rows, k, generator=g, device=DEV)).t
    ids = torch.randint(0, n, (rows, k), generator=g, device=DEV)
    if repeat and k > 2:
        ids[:, 2] = ids[:, 0]
    if gaps:
        ids[torch.rand(rows, k, generator=g, device=DEV) < 0.2] = -3
        top[torch.rand(rows, k, generator=g, device=DEV) < 0.1] = -math.inf
        if rows > 3:
            ids[3] = -1
    return top, ids


def check_distill(x, top, ids, temp, soft, targets, hard, weight, scale, dtype):
    t = x.shape[0]
    loss, d, alone = Vec(t), grad_of(x), Vec(t)
    args = (z.mat(x), z.mat(top) if top is not None else None, z.ids(ids) if ids is not None else None, temp, soft,
            z.ids(targets) if targets is not None else None, hard, weight, scale)
    z.zero_distill_loss(*args, loss.v, z.mat(d.t))
    w = weight
    if weight is not None and targets is not None:
        w = torch.where(targets < 0, torch.zeros_like(weight), weight)
    want_loss, want_grad = ref.distill(x, top, ids, temp, soft, targets, hard, w, scale, dtype)
    near(loss.v, want_loss, "loss")
    near(d.t, want_grad, "d_logits")
    loss.check()
    d.check()
    z.zero_distill_loss(*args, alone.v, None)
    assert torch.equal(alone.v, loss.v)
    d2 = grad_of(x)
    z.zero_distill_loss(*args, None, z.mat(d2.t))
    assert torch.equal(d2.t.nan_to_num(7), d.t.nan_to_num(7))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_cross_entropy(dtype, rows, vocab):
    g, x, targets = batch(3 * rows + vocab, rows, vocab, dtype)
    check_distill(x, None, None, 1.0, 0.0, targets, 1.0, None, 64.0 / rows, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (5, 9, 3), (33, 63, 17), (4, 1000, 256), (7, 4097, 64), (700, 257, 5),
                                          (9, 50257, 32), (2, 131079, 100), (2, 393211, 8)])
@pytest.mark.parametrize("temp,soft,hard", [(1.0, 1.0, 0.0), (2.0, 1.0, 0.0), (1.0, 0.7, 0.3), (2.0, 0.5, 0.5), (4.0, 0.5, 0.5),
                                            (3.3, 0.25, 0.75)])
def test_distillation(dtype, rows, vocab, k, temp, soft, hard):
    g, x, targets = batch(rows + 2 * vocab + k, rows, vocab, dtype)
    top, ids = teacher(g, x, k)
    weight = 0.5 + torch.rand(rows, generator=g, device=DEV)
    weight[targets < 0] = math.nan
    if k > 1 and vocab > 10:
        ids[:, 1] = targets               # the target among the teacher's entries
    check_distill(x, top, ids, temp, soft, targets, hard, weight, 8.0, dtype)


def test_distillation_without_targets():
    g, x, _ = batch(31, 45, 777, "f16", pad=0.0)
    top, ids = teacher(g, x, 12)
    check_distill(x, top, ids.int(), 2.0, 1.0, None, 0.0, None, 4.0, "f16")


def test_teacher_entries_beyond_the_vocabulary_and_special_logits():
    g, x, targets = batch(32, 6, 500, "bf16", pad=0.0)
    top, ids = teacher(g, x, 9, gaps=False)
    ids[1, 4], ids[2, 0] = 500, 1 << 33
    want = torch.where(ids < 500, ids, torch.full_like(ids, -1))
    out = []
    for i, flagged in ((ids, 1), (want, 0)):
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        loss, d = torch.empty(6, device=DEV), grad_of(x).t
        z.zero_distill_loss(z.mat(x), z.mat(top), z.ids(i), 1.0, 1.0, z.ids(targets), 0.5, None, 1.0, loss, z.mat(d), bad)
        assert int(bad) == flagged
        out.append((loss, d))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    # the student cannot choose an entry that the teacher does: an infinite loss, a finite gradient
    x[0, ids[0, 5]] = -math.inf
    targets[0] = (ids[0, 5] + 1) % 500
    top[3, 2] = math.nan
    loss, d = torch.empty(6, device=DEV), grad_of(x).t
    z.zero_distill_loss(z.mat(x), z.mat(top), z.ids(want), 1.0, 1.0, z.ids(targets), 0.5, None, 1.0, loss, z.mat(d))
    assert float(loss[0]) == math.inf and bool(torch.isfinite(d[0].float()).all())
    assert bool(torch.isnan(loss[3])) and bool(torch.isnan(d[3].float()).any())
    assert bool(torch.isfinite(loss[4:]).all())


# -- policy loss ------------------------------------------------------------------------


def policy_inputs(seed, rows, vocab, dtype, temp):
    g, x, targets = batch(seed, rows, vocab, dtype)
    r = ref.Rows(x, targets.clamp(min=0), temp, targets >= 0)
    lp = r.masked(r.lp).float()
    step = 0.3 * torch.randn(rows, generator=g, device=DEV)
    for border in (math.log(0.8), math.log(1.28), 0.0):
        step = torch.where((step - border).abs() < 1e-2, step + 3e-2, step)   # where either side may be taken
    gone = targets < 0
    old, rf = lp - step, lp + vec(g, rows, 0.4)
    adv, weight = vec(g, rows, 1.0), 0.3 + torch.rand(rows, generator=g, device=DEV)
    for v in (old, rf, adv, weight):
        v[gone] = math.nan
    return x, targets, old, rf, adv, weight


def clean(v, targets):
    return None if v is None else torch.where(targets < 0, torch.zeros_like(v), v)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("temp,kl,weighted", [(1.0, 0.0, False), (0.7, 0.1, True)])
def test_policy(dtype, rows, vocab, temp, kl, weighted):
    x, targets, old, rf, adv, weight = policy_inputs(rows + 5 * vocab, rows, vocab, dtype, temp)
    weight = weight if weighted else None
    loss, lp, d, alone = Vec(rows), Vec(rows), grad_of(x), Vec(rows)
    args = (z.mat(x), z.ids(targets), temp, old, rf if kl else None, adv, weight, 0.2, 0.28, kl, 16.0)
    z.zero_policy_loss(*args, loss.v, lp.v, z.mat(d.t))
    want = ref.policy(x, targets, temp, clean(old, targets), clean(rf, targets), clean(adv, targets),
                      clean(weight, targets), 0.2, 0.28, kl, 16.0, dtype)
    near(lp.v, want[1], "logp")
    near(loss.v, want[0], "loss")
    near(d.t, want[2], "d_logits")
    for b in (loss, lp, d):
        b.check()
    z.zero_policy_loss(*args, alone.v, None, None)
    assert torch.equal(alone.v, loss.v)


def test_policy_sides_of_the_clip():
    """Which rows have a gradient: none where the clipped value is the smaller, whatever its sign."""
    n = 64
    x = Banded(8, n, torch.float16, torch.zeros(8, n, device=DEV)).t
    targets = torch.arange(8, device=DEV)
    ratio = torch.tensor([1.0, 1.5, 0.5, 1.5, 0.5, 1.1, 0.9, 1.0], device=DEV)
    adv = torch.tensor([1.0, 1.0, 1.0, -1.0, -1.0, -2.0, 2.0, 0.0], device=DEV)
    old = -math.log(n) - torch.log(ratio)
    loss, d = Vec(8), grad_of(x)
    z.zero_policy_loss(z.mat(x), z.ids(targets), 1.0, old, None, adv, None, 0.2, 0.2, 0.0, 1.0, loss.v, None, z.mat(d.t))
    want = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv)
    assert torch.allclose(loss.v, want, rtol=1e-5, atol=0)
    has = d.t.abs().sum(1) > 0
    assert has.tolist() == [True, False, True, True, False, True, True, False]
    # nan advantages and log-probabilities of rows that count reach the gradient
    old[0] = math.nan
    adv[5] = math.nan
    z.zero_policy_loss(z.mat(x), z.ids(targets), 1.0, old, None, adv, None, 0.2, 0.2, 0.0, 1.0, loss.v, None, z.mat(d.t))
    for row in (0, 5):
        assert bool(torch.isnan(loss.v[row])) and bool(torch.isnan(d.t[row]).all())


def test_policy_close_to_the_reference():
    """The KL term where exp(d) - d - 1 would cancel."""
    n = 16
    x = Banded(40, n, torch.float16, torch.zeros(40, n, device=DEV)).t
    targets = torch.zeros(40, dtype=torch.int64, device=DEV)
    lp = torch.empty(40, device=DEV)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, lp)
    rf = lp + torch.logspace(-3, 0.3, 40, device=DEV)
    d = rf.double() - lp.double()
    loss = torch.empty(40, device=DEV)
    z.zero_policy_loss(z.mat(x), z.ids(targets), 1.0, lp, rf, torch.zeros(40, device=DEV), None, 0.2, 0.2, 1.0, 1.0, loss)
    want = torch.expm1(d) - d
    # d is exact here (both are of one binade or close to it), so only the series' and expm1's roundings count: at d = 0.3
    # expm1 and the difference lose a factor of 0.35 / 0.05
    assert bool(((loss.double() - want).abs() <= 2.0 ** -19 * want).all())


# -- preference loss -----------------------------------------------------------------


def starts_of(lengths, dtype=torch.int64):
    return torch.cumsum(torch.tensor([0] + list(lengths)), 0).to(dtype).to(DEV)


def check_preference(x, targets, starts, rf, beta, smoothing, scale, dtype):
    t, pairs = x.shape[0], starts.numel() // 2
    loss, reward, lp, d = Vec(pairs), Vec(2 * pairs), Vec(t), grad_of(x)
    ws = space(z.zero_preference_loss_workspace(t, pairs))
    args = (z.mat(x), z.ids(targets), z.ids(starts), rf, beta, smoothing, scale)
    z.zero_preference_loss(*args, loss.v, reward.v, lp.v, z.mat(d.t), ws, ws.numel())
    at = starts.tolist()
    rows = torch.arange(t, device=DEV)
    there = (targets >= 0) & (rows >= at[0]) & (rows < at[-1])
    safe = None if rf is None else torch.where(there, rf, torch.zeros_like(rf))
    want = ref.preference(x, targets, starts, safe, beta, smoothing, scale, dtype)
    near(loss.v, want[0], "loss")
    near(reward.v, want[1], "reward")
    near(lp.v, want[2], "logp")
    near(d.t, want[3], "d_logits")
    for b in (loss, reward, lp, d):
        b.check()
    alone = Vec(pairs)
    z.zero_preference_loss(*args, alone.v, None, None, None, ws, ws.numel())
    assert torch.equal(alone.v, loss.v)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,behind,vocab", [([1, 1], 0, 5), ([3, 4, 5, 6], 2, 1000), ([0, 7, 9, 0, 0, 0], 3, 63),
                                                  ([40, 33], 1, 50257), ([300, 1, 2, 500], 0, 257), ([5, 4], 0, 131079)])
@pytest.mark.parametrize("smoothing,has_ref", [(0.0, True), (0.2, False)])
def test_preference(dtype, lengths, behind, vocab, smoothing, has_ref):
    rows = sum(lengths) + behind
    g, x, targets = batch(rows * 3 + vocab, rows, vocab, dtype)
    rf = vec(g, rows, 1.0, targets < 0) - 5.0 if has_ref else None
    check_preference(x, targets, starts_of(lengths), rf, 0.1, smoothing, 32.0, dtype)


def test_preference_rows_before_and_behind():
    """Rows of no sequence are left out whatever they and their targets hold."""
    g, x, targets = batch(51, 30, 400, "f16", pad=0.0)
    starts = torch.tensor([4, 11, 25], dtype=torch.int32, device=DEV)
    x[:4], x[25:] = math.nan, math.inf
    targets[1], targets[27] = 1 << 20, 400
    rf = vec(g, 30) - 4
    rf[:4], rf[25:] = math.nan, math.nan
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_preference(x, targets.clamp(max=399), starts, rf, 0.5, 0.0, 1.0, "f16")
    loss, ws = torch.empty(1, device=DEV), space(z.zero_preference_loss_workspace(30, 1))
    d = grad_of(x).t
    z.zero_preference_loss(z.mat(x), z.ids(targets), z.ids(starts), rf, 0.5, 0.0, 1.0, loss, None, None, z.mat(d), ws,
                           ws.numel(), bad)
    assert int(bad) == 0 and bool((d[:4] == 0).all()) and bool((d[25:] == 0).all())


@pytest.mark.parametrize("numbers", [[0, 10, 5], [0, 10, 31], [-1, 10, 20], [5, 4, 20], [0, 10, 20, 15, 30], [0, 1 << 40, 30]])
def test_preference_starts_that_do_not_rise(numbers):
    g, x, targets = batch(52, 30, 100, "bf16", pad=0.0)
    starts = torch.tensor(numbers, device=DEV)
    pairs = len(numbers) // 2
    loss, reward, d = Vec(pairs), Vec(2 * pairs), grad_of(x)
    ws = space(z.zero_preference_loss_workspace(30, pairs))
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    z.zero_preference_loss(z.mat(x), z.ids(targets), z.ids(starts), None, 0.1, 0.0, 1.0, loss.v, reward.v, None, z.mat(d.t), ws,
                           ws.numel(), bad)
    assert int(bad) == 1
    assert bool(torch.isnan(loss.v[-1])) and bool(torch.isnan(reward.v[-2:]).all())
    assert bool(torch.isnan(d.t.float()).any())
    d.check()


def test_preference_extreme_margins():
    g, x, targets = batch(53, 8, 50, "bf16", pad=0.0)
    starts = starts_of([4, 4])
    for beta in (100.0, -100.0, 0.0):
        for smoothing in (0.0, 0.3, 1.0):
            check_preference(x, targets, starts, None, beta, smoothing, 1.0, "bf16")


# -- all of them ----------------------------------------------------------------------


def test_no_rows():
    x = torch.empty(0, 100, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    e = torch.empty(0, device=DEV)
    z.zero_token_logprob(z.mat(x), z.ids(none), 1.0, torch.empty(1, device=DEV))
    z.zero_token_logprob_backward(z.mat(x), z.ids(none), 1.0, e, z.mat(x))
    z.zero_distill_loss(z.mat(x), None, None, 1.0, 0.0, z.ids(none), 1.0, None, 1.0, torch.empty(1, device=DEV), None)
    z.zero_policy_loss(z.mat(x), z.ids(none), 1.0, e, None, e, None, 0.2, 0.2, 0.0, 1.0, torch.empty(1, device=DEV))
    loss, reward = torch.empty(2, device=DEV), torch.empty(4, device=DEV)
    ws = space(z.zero_preference_loss_workspace(0, 2))
    z.zero_preference_loss(z.mat(x), z.ids(none), z.ids(torch.zeros(5, dtype=torch.int64, device=DEV)), None, 0.1, 0.0, 1.0, loss,
                           reward, None, z.mat(x), ws, ws.numel())
    assert bool(((loss - math.log(2.0)).abs() < 1e-6).all()) and bool((reward == 0).all())


def test_rows_of_no_pair():
    _, x, targets = batch(61, 9, 40, "f16", pad=0.0)
    d, lp = grad_of(x), Vec(9)
    ws = space(z.zero_preference_loss_workspace(9, 0))
    z.zero_preference_loss(z.mat(x), z.ids(targets), z.ids(torch.zeros(1, dtype=torch.int64, device=DEV)), None, 0.1, 0.0, 1.0,
                           None, None, lp.v, z.mat(d.t), ws, ws.numel())
    assert bool((d.t == 0).all()) and bool((lp.v == 0).all())
    d.check()


@pytest.mark.parametrize("pad", [0.0, 1.0])
def test_every_row_padded_or_none(pad):
    g, x, targets = batch(62, 20, 600, "bf16", pad=pad)
    check_distill(x, None, None, 1.0, 0.0, targets, 1.0, None, 1.0, "bf16")


def calls(seed, dtype, rows, vocab):
    """Every operator once over the same rows: (its call, its outputs)."""
    g, x, targets = batch(seed, rows, vocab, dtype)
    top, ids = teacher(g, x, 12)
    old = vec(g, rows) - 6
    pairs = 2
    starts = starts_of([rows // 4, rows // 4, rows // 4, rows // 8])
    f = lambda n: torch.empty(n, device=DEV)                               # noqa: E731
    lp, lse, l1, l2, l3, lp2, rew = f(rows), f(rows), f(rows), f(rows), f(pairs), f(rows), f(2 * pairs)
    d = [torch.empty(rows, -(-vocab // 8) * 8, dtype=x.dtype, device=DEV)[:, :vocab] for _ in range(4)]
    ws = space(z.zero_preference_loss_workspace(rows, pairs))
    m, t = z.mat(x), z.ids(targets)

    def run(st=None):
        z.zero_token_logprob(m, t, 1.0, lp, lse, stream=st)
        z.zero_token_logprob_backward(m, t, 1.0, old, z.mat(d[0]), stream=st)
        z.zero_distill_loss(m, z.mat(top), z.ids(ids), 2.0, 0.5, t, 0.5, None, 8.0, l1, z.mat(d[1]), stream=st)
        z.zero_policy_loss(m, t, 1.0, old, lp, old, None, 0.2, 0.2, 0.1, 8.0, l2, lp2, z.mat(d[2]), stream=st)
        z.zero_preference_loss(m, t, z.ids(starts), old, 0.1, 0.1, 8.0, l3, rew, None, z.mat(d[3]), ws, ws.numel(), stream=st)

    return run, [lp, lse, l1, l2, l3, lp2, rew, *d], (x, targets, top, ids, old, starts, ws)


@pytest.mark.parametrize("rows,vocab", [(64, 777), (1000, 5000), (40, 50257)])
def test_results_repeat_on_another_stream_and_in_a_graph(rows, vocab):
    run, outs, _keep = calls(71, "bf16", rows, vocab)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]

    def same():
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a.nan_to_num(5), b.nan_to_num(5))
            a.fill_(3)
        torch.cuda.synchronize()

    same()
    run()
    run()
    same()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(side)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        same()


def test_two_streams_at_once():
    """Calls that run at the same time, each with its own outputs and workspace."""
    a, outs_a, _ka = calls(81, "f16", 300, 3001)
    b, outs_b, _kb = calls(82, "bf16", 256, 9000)
    a()
    b()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs_a + outs_b]
    for o in outs_a + outs_b:
        o.fill_(3)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        a(s)
        b(t)
    torch.cuda.synchronize()
    for o, w in zip(outs_a + outs_b, want):
        assert torch.equal(o.nan_to_num(5), w.nan_to_num(5))


def test_offsets_beyond_32_bits():
    """Rows whose elements lie beyond 2^32 of the matrix's start."""
    rows, vocab = 90000, 50000
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    targets = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
    g = gen(91)
    at = torch.tensor([0, 1, 42949, 42950, 85899, 85900, rows - 1], device=DEV)
    x[at] = (2 * torch.randn(len(at), vocab, generator=g, device=DEV)).to(x.dtype)
    targets[at] = torch.randint(0, vocab, (len(at),), generator=g, device=DEV)
    lp = torch.empty(rows, device=DEV)
    z.zero_token_logprob(z.mat(x), z.ids(targets), 1.0, lp)
    r = ref.Rows(x[at], targets[at], 1.0, torch.ones(len(at), dtype=torch.bool, device=DEV))
    near(lp[at], (r.lp, r.lp_tol), "logp")
    one = torch.ones(rows, device=DEV)
    want = ref.logprob_backward(x[at], targets[at], 1.0, one[at], "bf16")
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, one, z.mat(x))
    near(x[at], want, "d_logits")
    others = torch.ones(rows, dtype=torch.bool, device=DEV)
    others[at] = False
    assert float(lp[others].abs().max()) == 0.0
    for a in range(0, rows, 10000):
        part = x[a:a + 10000][others[a:a + 10000]]
        assert not bool(part.any())


def test_scoring_then_policy_and_pair_steps():
    """The operators together as a program uses them: the frozen and the sampling model score a batch, the policy step
    and the preference step take those scores; at the same parameters the ratio is 1, and the margin is 0."""
    g, x, targets = batch(95, 120, 3001, "f16")
    old, frozen = torch.empty(120, device=DEV), torch.empty(120, device=DEV)
    m, t = z.mat(x), z.ids(targets)
    z.zero_token_logprob(m, t, 1.0, old)
    z.zero_token_logprob(m, t, 1.0, frozen)
    adv = vec(g, 120)
    loss, lp, d = torch.empty(120, device=DEV), torch.empty(120, device=DEV), grad_of(x)
    z.zero_policy_loss(m, t, 1.0, old, frozen, adv, None, 0.2, 0.2, 0.1, 4.0, loss, lp, z.mat(d.t))
    # the two log-probabilities are sums of the same numbers in two orders
    live = targets >= 0
    r = ref.Rows(x, targets.clamp(min=0), 1.0, live)
    tol = 2 * r.masked(r.lp_tol)
    assert bool(((lp.double() - old.double()).abs() <= tol).all())
    # so the ratio is 1 and the KL term's slope 0 to within that; 0.1 is its weight
    assert bool(((loss.double() + adv.double()).abs()[live] <= (adv.double().abs() * (tol + 2.0 ** -21) + 0.1 * tol)[live]).all())
    want = ref.logprob_backward(x, targets, 1.0, -4.0 * adv, "f16")
    extra = 4.0 * (adv.double().abs() * (tol + 2.0 ** -21) + 0.1 * (tol + 2.0 ** -21))[:, None] * (r.p.nan_to_num(0) + 1)
    near(d.t, (want[0], want[1] + r.masked(extra)), "d_logits")
    starts = starts_of([30, 30, 20, 40])
    pl, rew, ws = torch.empty(2, device=DEV), torch.empty(4, device=DEV), space(z.zero_preference_loss_workspace(120, 2))
    z.zero_preference_loss(m, t, z.ids(starts), frozen, 0.1, 0.0, 4.0, pl, rew, None, z.mat(d.t), ws, ws.numel())
    # the sums take the policy's log-probabilities unrounded, and the frozen model's as they are given: each is off by
    # half a step of fp32 at most; and they may be sums in two orders
    off = [0.1 * float((2.0 ** -24 * frozen.double().abs() + tol)[a:b].sum()) for a, b in zip(starts.tolist(), starts.tolist()[1:])]
    assert all(abs(r) <= o + 1e-12 for r, o in zip(rew.tolist(), off))
    assert bool(((pl - math.log(2.0)).abs() < 1e-6 + sum(off)).all())
    slope = torch.zeros(120, device=DEV)
    for i, (a, b) in enumerate(zip(starts.tolist(), starts.tolist()[1:])):
        slope[a:b] = -0.05 * 4.0 if i % 2 == 0 else 0.05 * 4.0
    want = ref.logprob_backward(x, targets, 1.0, slope, "f16")
    near(d.t, (want[0], want[1] + r.masked(4.0 * 0.1 * sum(off) * (r.p.nan_to_num(0) + 1))), "d_logits")


# -- every instance -----------------------------------------------------------------------

# (rows, vocabulary, layouts of the gradient, with a teacher, of the scores): loss_rule
MANY = [(700, 40), (700, 4096), (640, 4100), (620, 8300), (610, 32001), (615, 50257), (609, 57000), (612, 100003),
        (609, 114001), (620, 131072)]
FEW = [(3, 300), (150, 600), (20, 4100), (9, 8300), (30, 32001), (300, 20000), (64, 57000), (1, 114001), (7, 131072)]


def test_the_sizes_run_every_layout():
    seen = {kind: {rule.layout(r, v, *kind) for r, v in MANY + FEW} for kind in ((True, False), (True, True), (False, False))}
    for kind, layouts in seen.items():
        assert {t for t, _ in layouts} == {32, 128, 256, 512}, (kind, layouts)
        assert {1, 2, 4, 5, 8} <= {c for _, c in layouts}, (kind, layouts)
    # over clusters, many rows: a CTA takes several, by turns
    for kind in seen:
        assert any(rule.layout(r, v, *kind)[1] > 1 for r, v in MANY)


@pytest.mark.parametrize("dtype,rows,vocab", [(DTYPES[i % 2], *s) for i, s in enumerate(MANY + FEW)])
def test_layouts(dtype, rows, vocab):
    g, x, targets = batch(rows + vocab, rows, vocab, dtype, pad=0.3)
    check_logprob(x, targets, 1.3)
    check_distill(x, None, None, 1.0, 0.0, targets, 1.0, None, 2.0, dtype)
    torch.cuda.empty_cache()
    top, ids = teacher(g, x, 19)
    ids[:, 1] = targets
    for temp in (2.0, 3.0):
        check_distill(x, top, ids, temp, 0.5, targets, 0.5, None, 2.0, dtype)
        torch.cuda.empty_cache()
    d_lp = vec(g, rows, 1.0, targets < 0)
    d = grad_of(x)
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, d_lp, z.mat(d.t))
    z.zero_token_logprob_backward(z.mat(x), z.ids(targets), 1.0, d_lp, z.mat(x))
    assert torch.equal(x, d.t)


@pytest.mark.parametrize("rows,vocab", [(700, 257), (640, 5000), (615, 50257)])
@pytest.mark.parametrize("temp", [1.0, 2.0, 4.0, 2.7])
def test_many_rows_with_the_most_entries(rows, vocab, temp):
    g, x, targets = batch(rows, rows, vocab, "bf16", pad=0.5)
    top, ids = teacher(g, x, 256)
    check_distill(x, top, ids, temp, 0.75, targets, 0.25, None, 4.0, "bf16")


@pytest.mark.parametrize("rows,vocab", [(700, 257), (640, 5000), (615, 50257), (612, 100003)])
def test_many_rows_in_pairs(rows, vocab):
    g, x, targets = batch(rows, rows, vocab, "f16", pad=0.3)
    lengths = [rows // 5, rows // 7, 0, rows // 3, 1, 1]
    check_preference(x, targets, starts_of(lengths), vec(g, rows, 1.0, targets < 0) - 5, 0.1, 0.1, 16.0, "f16")


def test_logits_that_lie_apart_on_lines():
    """Rows on every 16-byte boundary of a 128-byte line, and gradients on another than the logits."""
    rows, vocab = 640, 4111
    g, x, targets = batch(77, rows, vocab, "f16")
    buf = torch.empty(64 + rows * 4136, dtype=torch.float16, device=DEV)
    for off in (0, 8, 24, 56):
        y = buf[off:off + rows * 4136].view(rows, 4136)[:, :vocab]        # rows 4,136 * 2 = 64 * 129 + 16 bytes apart
        y.copy_(x)
        loss, d = torch.empty(rows, device=DEV), grad_of(x)
        z.zero_distill_loss(z.mat(y), None, None, 1.0, 0.0, z.ids(targets), 1.0, None, 1.0, loss, z.mat(d.t))
        want_loss, want = ref.distill(y, None, None, 1.0, 0.0, targets, 1.0, None, 1.0, "f16")
        near(loss, want_loss, "loss")
        near(d.t, want, "d_logits")
        d.check()
