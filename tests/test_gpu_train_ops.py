"""The training operators on the GPU against their definitions in 64 bits, at
the sizes, strides and values where they can go wrong.  The bounds are those
of the roundings the operators document (train_ref)."""
import pytest
import torch

import train_ref as ref
import zero_sharded_optimizer_02_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = ["f16", "bf16"]


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

    def __init__(self, rows, cols, dtype, pitch=None, offset=0, fill=None):
        self.pitch = pitch if pitch is not None else -(-cols // 16) * 16 + 16
        n = 64 + offset + rows * self.pitch + 64
        self.buf = torch.full((n,), 77, dtype=dtype, device=DEV)
        self.t = self.buf[64 + offset:64 + offset + rows * self.pitch].view(rows, self.pitch)[:, :cols]
        if fill is not None:
            self.t.copy_(fill)
        self.before = self.buf.clone()

    def check(self, what):
        now = self.buf.clone()
        inside = torch.zeros_like(now, dtype=torch.bool)
        torch.as_strided(inside, self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(True)
        assert torch.equal(now[~inside], self.before[~inside]), f"{what}: written outside its elements"


def act(g, rows, cols, dtype, sigma=1.0, big=0.0):
    x = torch.randn(rows, cols, generator=g, device=DEV) * sigma
    if big and cols > 3:
        x[:, 3::37] *= big
    return Banded(rows, cols, ref.TYPES[dtype], fill=x).t


def workspace(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)


# -- 8-bit checkpoints ------------------------------------------------------------


def new_act8(rows, cols):
    q = Banded(rows, cols, torch.int8, pitch=-(-cols // 16) * 16 + 16)
    s = Banded(rows, -(-cols // 32), torch.uint8, pitch=-(-cols // 32) + 3)
    return q, s


def check_pack(x, dtype):
    rows, cols = x.shape
    q, s = new_act8(rows, cols)
    z.zero_act_pack(z.mat(x), z.act8(q.t, s.t))
    rq, rs = ref.pack(x, dtype)
    assert torch.equal(s.t.cpu(), rs), "scale bytes"
    assert torch.equal(q.t.cpu(), rq), "elements"
    q.check("q")
    s.check("scale")
    out = Banded(rows, cols, ref.TYPES[dtype])
    z.zero_act_unpack(z.act8(q.t, s.t), z.mat(out.t))
    v = ref.values(rq, rs)
    assert torch.equal(torch.isnan(out.t.cpu()), torch.isnan(v))
    ok = ~torch.isnan(v)
    assert torch.equal(out.t.cpu().double()[ok], v[ok]), "read back"   # exact in the type
    out.check("unpacked")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 32), (7, 33), (2, 8), (33, 1111),
                                       (64, 1600), (1025, 96), (3, 40000)])
def test_pack_and_unpack(dtype, rows, cols):
    check_pack(act(gen(rows * 1000 + cols), rows, cols, dtype, 3.0, 50.0), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_every_encoding(dtype):
    """All 65,536 encodings (subnormals, the largest, infinities and NaNs), in
    blocks of alike and of mixed magnitudes."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(ref.TYPES[dtype]).reshape(64, 1024).to(DEV)
    check_pack(x, dtype)
    check_pack(x.t().contiguous(), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_special_blocks(dtype):
    t = ref.TYPES[dtype]
    top = torch.finfo(t).max
    x = torch.zeros(8, 72, dtype=t, device=DEV)[:, :70]
    x[1] = top
    x[2, 5], x[2, 40] = float("inf"), 1.0
    x[3, 69] = float("nan")
    x[4] = torch.finfo(t).tiny / 2
    x[5, 0] = -top
    x[6, 31:33] = torch.tensor([127.0, 254.0], dtype=t)
    x[7, ::2] = -127.5 if dtype == "f16" else -127.0
    check_pack(x, dtype)


def test_unpack_into_the_other_type():
    """A bfloat16 checkpoint read as binary16 rounds once, past its range to inf."""
    x = act(gen(5), 9, 77, "bf16", 1e4, 100.0)
    q, s = z.act8_empty(9, 77)
    z.zero_act_pack(z.mat(x), z.act8(q, s))
    out = torch.empty(9, 80, dtype=torch.float16, device=DEV)[:, :77]
    z.zero_act_unpack(z.act8(q, s), z.mat(out))
    assert torch.equal(out.cpu(), ref.values(q.cpu(), s.cpu()).to(torch.float16))


# -- norm --------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 1600), (3, 33), (5, 8), (17, 768), (2, 2056), (9, 4096), (3, 8200),
               (2, 32768), (300, 160), (700, 257), (2047, 1601)]


def check_checkpoint(q, s, xhat, dtype, what):
    """Every value within half a step of xhat; every step the least that fits (both up to fp32)."""
    lo, hi = ref.LIMITS[dtype]
    v = ref.values(q, s)
    step = ref.two_to(s.long() - 127)[:, torch.arange(q.shape[1], device=q.device) // ref.BLOCK]
    ref.assert_within(v, xhat, 0.5 * step + 1e-5 * xhat.abs(), what)
    nb = s.shape[1]
    pad = torch.nn.functional.pad(xhat, (0, nb * ref.BLOCK - xhat.shape[1]))
    a = pad.view(-1, nb, ref.BLOCK).abs().amax(2)
    step = ref.two_to(s.long() - 127)
    assert bool((a <= 127 * step * (1 + 1e-5)).all()), f"{what}: a step too small"
    assert bool(((a >= 63.5 * step * (1 - 1e-5)) | (s.long() - 127 == lo)).all()), f"{what}: a step too large"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("residual,gain", [(True, True), (False, False)])
def test_norm_forward(dtype, rows, cols, residual, gain):
    g = gen(rows + 7 * cols)
    t = ref.TYPES[dtype]
    x = act(g, rows, cols, dtype, 0.5)
    res = act(g, rows, cols, dtype, 2.0, 12.0) if residual else None
    # a gain that starts 2 bytes past a 16-byte boundary, as in a flat buffer
    w = (1 + 0.2 * torch.randn(cols + 1, generator=g, device=DEV)).to(t)[1:] if gain else None
    h, y = Banded(rows, cols, t), Banded(rows, cols, t)
    rstd = Banded(1, rows, torch.float32)
    q, s = new_act8(rows, cols)
    z.zero_norm_forward(z.mat(x), z.mat(res) if residual else None, w, 1e-5, z.mat(h.t), z.mat(y.t),
                        rstd.t, z.act8(q.t, s.t))
    h64, r64, xhat, y64 = ref.norm_forward(x, res, w, 1e-5)
    fp = (cols + 16) * ref.E32
    ref.assert_within(h.t, h64, (ref.U[dtype] + 2 * ref.E32) * h64.abs() + ref.TINY[dtype], "h")
    ref.assert_within(rstd.t[0], r64, fp * r64, "rstd")
    ref.assert_within(y.t, y64, (ref.U[dtype] + 2 * fp) * y64.abs() + ref.TINY[dtype], "y")
    check_checkpoint(q.t, s.t, xhat, dtype, "checkpoint")
    for b, name in ((h, "h"), (y, "y"), (rstd, "rstd"), (q, "q"), (s, "scale")):
        b.check(name)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_forward_outputs_one_by_one_and_in_place(dtype):
    rows, cols = 37, 1000
    g = gen(3)
    t = ref.TYPES[dtype]
    x, res = act(g, rows, cols, dtype), act(g, rows, cols, dtype, 2.0)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(t)
    new = lambda: Banded(rows, cols, t).t  # noqa: E731
    h, y, rstd = new(), new(), torch.empty(rows, device=DEV)
    q, s = z.act8_empty(rows, cols)
    z.zero_norm_forward(z.mat(x), z.mat(res), w, 1e-5, z.mat(h), z.mat(y), rstd, z.act8(q, s))
    y1, r1, (q1, s1) = new(), torch.empty(rows, device=DEV), z.act8_empty(rows, cols)
    z.zero_norm_forward(z.mat(x), z.mat(res), w, 1e-5, None, z.mat(y1))
    z.zero_norm_forward(z.mat(x), z.mat(res), w, 1e-5, None, None, r1)
    z.zero_norm_forward(z.mat(x), z.mat(res), w, 1e-5, None, None, None, z.act8(q1, s1))
    assert torch.equal(y1, y) and torch.equal(r1, rstd)
    assert torch.equal(q1, q) and torch.equal(s1, s)
    for into in ("x", "res"):   # h takes the place of one of its inputs
        a = {"x": Banded(rows, cols, t, fill=x), "res": Banded(rows, cols, t, fill=res)}
        z.zero_norm_forward(z.mat(a["x"].t), z.mat(a["res"].t), w, 1e-5, z.mat(a[into].t), None)
        assert torch.equal(a[into].t, h)
        a[into].check(into)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_zero_and_nonfinite_rows(dtype):
    rows, cols = 6, 100
    t = ref.TYPES[dtype]
    x = torch.zeros(rows, 104, dtype=t, device=DEV)[:, :cols]
    x[1, 50] = float("nan")
    x[2, 99] = float("inf")
    x[3] = 1.0
    x[4] = torch.finfo(t).tiny
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    q, s = z.act8_empty(rows, cols)
    y = torch.empty(rows, 104, dtype=t, device=DEV)[:, :cols]
    z.zero_norm_forward(z.mat(x), None, None, 1e-5, None, z.mat(y), rstd, z.act8(q, s))
    assert not y[0].any() and not q[0].any() and float(rstd[0]) == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    assert bool(torch.isnan(y[1]).all()) and bool((s[1] == 255).all())
    # an infinity: its row's rstd is 0, the element itself and its block are lost
    assert bool(torch.isnan(y[2, 99])) and int(s[2, 3]) == 255 and not y[2, :96].any()
    assert bool(torch.isfinite(y[3:]).all()) and bool((s[3:] != 255).all())
    # the gradient of a row with a lost block is NaN throughout, and so is the gain's
    dy = torch.ones(rows, 104, dtype=t, device=DEV)[:, :cols]
    dx = torch.empty(rows, 104, dtype=t, device=DEV)[:, :cols]
    dg = torch.zeros(cols, dtype=t, device=DEV)
    ws = workspace(z.zero_norm_backward_workspace(rows, cols))
    z.zero_norm_backward(z.mat(dy), z.act8(q, s), rstd, None, None, z.mat(dx), dg, False, ws, ws.numel())
    assert bool(torch.isnan(dx[1]).all()) and bool(torch.isnan(dx[2]).all())
    assert bool(torch.isfinite(dx[[0, 3, 4, 5]]).all())
    assert bool(torch.isnan(dg).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("residual,gain,add", [(True, True, False), (False, False, True)])
def test_norm_backward(dtype, rows, cols, residual, gain, add):
    g = gen(rows * 3 + cols)
    t = ref.TYPES[dtype]
    q, s = z.act8_empty(rows, cols)
    hsrc, rstd = act(g, rows, cols, dtype, 2.0, 12.0), torch.empty(rows, device=DEV)
    z.zero_norm_forward(z.mat(hsrc), None, None, 1e-5, None, None, rstd, z.act8(q, s))
    dy = act(g, rows, cols, dtype, 0.1)
    dres = act(g, rows, cols, dtype, 0.1) if residual else None
    w = (1 + 0.2 * torch.randn(cols + 1, generator=g, device=DEV)).to(t)[1:] if gain else None
    old = torch.randn(1, cols, generator=g, device=DEV).to(t)
    dx, dg = Banded(rows, cols, t), Banded(1, cols, t, offset=1, fill=old)   # odd 2-byte offset
    ws = workspace(z.zero_norm_backward_workspace(rows, cols))
    z.zero_norm_backward(z.mat(dy), z.act8(q, s), rstd, w, z.mat(dres) if residual else None,
                         z.mat(dx.t), dg.t, add, ws, ws.numel())
    xhat = ref.values(q, s)
    dx64, dg64, err, size = ref.norm_backward(dy, xhat, rstd, w, dres)
    u = ref.U[dtype]
    ref.assert_within(dx.t, dx64, u * (dx64.abs() + err) + err + ref.TINY[dtype], "dx")
    if add:
        dg64, size = dg64 + old[0].double(), size + old[0].double().abs()
    err = (rows + 8) * ref.E32 * size
    ref.assert_within(dg.t[0], dg64, u * (dg64.abs() + err) + err + ref.TINY[dtype], "d_gain")
    dx.check("dx")
    dg.check("d_gain")
    # without a gain gradient, and in place of dy: the same dx
    again = Banded(rows, cols, t, fill=dy)
    z.zero_norm_backward(z.mat(again.t), z.act8(q, s), rstd, w, z.mat(dres) if residual else None,
                         z.mat(again.t), None, False, None, 0)
    assert torch.equal(again.t, dx.t)
    # in place of the residual's gradient, another run of the same sums: the same bits
    dg2 = Banded(1, cols, t, offset=1, fill=old)
    into = Banded(rows, cols, t, fill=dres if residual else torch.zeros_like(dy))
    z.zero_norm_backward(z.mat(dy), z.act8(q, s), rstd, w, z.mat(into.t) if residual else None,
                         z.mat(into.t), dg2.t, add, ws, ws.numel())
    assert torch.equal(into.t, dx.t) and torch.equal(dg2.t, dg.t)


def test_norm_gradient_against_differences():
    """The definition's gradient against central differences in 64 bits, then the
    kernels' against the differences within what the 8-bit checkpoint and one
    rounding allow."""
    rows, cols, eps = 4, 96, 1e-5
    g = gen(11)
    x, dy = act(g, rows, cols, "f16"), act(g, rows, cols, "f16", 0.1)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(torch.float16)
    loss = lambda a, b: float((ref.norm_forward(a, None, b, eps)[3] * dy.double()).sum())  # noqa: E731
    _, r64, xhat, _ = ref.norm_forward(x, None, w, eps)
    dx64, dg64, _, _ = ref.norm_backward(dy, xhat, r64, w, None)
    q, s = z.act8_empty(rows, cols)
    rstd, dx, dg = torch.empty(rows, device=DEV), torch.empty_like(dy), torch.empty_like(w)
    z.zero_norm_forward(z.mat(x), None, w, eps, None, None, rstd, z.act8(q, s))
    dx = torch.empty(rows, cols, dtype=torch.float16, device=DEV)
    ws = workspace(z.zero_norm_backward_workspace(rows, cols))
    z.zero_norm_backward(z.mat(dy), z.act8(q, s), rstd, w, None, z.mat(dx), dg, False, ws, ws.numel())
    off = (ref.values(q, s) - xhat).abs()          # what the checkpoint lost
    u = (dy.double() * w.double()).abs()
    for k in range(6):
        d = torch.randn(rows, cols, generator=g, device=DEV).double()
        step = 1e-6
        num = (loss(x.double() + step * d, w) - loss(x.double() - step * d, w)) / (2 * step)
        assert float((dx64 * d).sum()) == pytest.approx(num, rel=1e-6, abs=1e-6)
        lost = r64[:, None] * (off * (u * xhat.abs()).mean(1, keepdim=True) +
                               (xhat.abs() + off) * (u * off).mean(1, keepdim=True))
        bound = float(((lost + 2 * ref.U["f16"] * dx64.abs() + 1e-6) * d.abs()).sum())
        assert abs(float((dx.double() * d).sum()) - num) <= bound
        e = torch.randn(cols, generator=g, device=DEV).double()
        num = (loss(x.double(), w.double() + step * e) - loss(x.double(), w.double() - step * e)) / (2 * step)
        assert float((dg64 * e).sum()) == pytest.approx(num, rel=1e-6, abs=1e-6)
        bound = float((((dy.double().abs() * off).sum(0) + 2 * ref.U["f16"] * dg64.abs() + 1e-6) * e.abs()).sum())
        assert abs(float((dg.double() * e).sum()) - num) <= bound


# -- embedding -----------------------------------------------------------------------


def table_of(g, vocab, dim, dtype, flat_offset=0, pitch=None):
    """A table inside a flat buffer, at any 2-byte offset."""
    return Banded(vocab, dim, ref.TYPES[dtype], pitch=pitch or dim, offset=flat_offset,
                  fill=torch.randn(vocab, dim, generator=g, device=DEV) * 0.5)


EMBED_SHAPES = [(1, 1, 1), (1, 50257, 768), (7, 3, 33), (1021, 997, 64), (5000, 300, 40),
                (2048, 65, 264), (4097, 70000, 24)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,vocab,dim", EMBED_SHAPES)
@pytest.mark.parametrize("offset,id_type", [(0, torch.int64), (3, torch.int32)])
def test_embed_lookup(dtype, tokens, vocab, dim, offset, id_type):
    g = gen(tokens + vocab)
    table = table_of(g, vocab, dim, dtype, offset)
    ids = torch.randint(-1, vocab, (tokens,), generator=g, device=DEV).to(id_type)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    for scale in (1.0, -40.0):
        out = Banded(tokens, dim, ref.TYPES[dtype])
        z.zero_embed_lookup(z.mat(table.t), z.ids(ids), scale, z.mat(out.t), bad)
        want = (table.t[ids.long().clamp(min=0)].float() * scale).to(ref.TYPES[dtype])
        want[ids < 0] = 0
        assert torch.equal(out.t, want)
        out.check("lookup")
    assert int(bad) == 0
    if tokens > 1:
        ids[tokens // 2] = vocab
        z.zero_embed_lookup(z.mat(table.t), z.ids(ids), 1.0, z.mat(out.t), bad)
        assert int(bad) == 1 and not out.t[tokens // 2].any()
        z.zero_embed_lookup(z.mat(table.t), z.ids(ids), 1.0, z.mat(out.t))   # no flag wanted


def run_embed_grad(d_out, ids, scale, add, table, bad=None):
    ws = workspace(z.zero_embed_grad_workspace(ids.numel(), table.t.shape[0], table.t.shape[1]))
    z.zero_embed_grad(z.mat(d_out), z.ids(ids), scale, add, z.mat(table.t), ws, ws.numel(), bad)


def check_embed_grad(d_out, ids, scale, add, vocab, dtype, offset=0, pitch=None, seed=0):
    g = gen(seed)
    dim = d_out.shape[1]
    table = table_of(g, vocab, dim, dtype, offset, pitch)
    old = table.t.clone()
    run_embed_grad(d_out, ids, scale, add, table)
    total, size, count = ref.embed_grad(d_out, ids, scale, vocab, old if add else None)
    err = (count + 3)[:, None] * ref.E32 * size
    ref.assert_within(table.t, total, ref.U[dtype] * (total.abs() + err) + err + ref.TINY[dtype], "d_table")
    table.check("d_table")
    absent = count == 0
    assert torch.equal(table.t[absent], old[absent] if add else torch.zeros_like(old[absent]))
    again = Banded(vocab, dim, ref.TYPES[dtype], pitch=pitch or dim, offset=offset, fill=old)
    run_embed_grad(d_out, ids, scale, add, again)
    assert torch.equal(again.t, table.t), "two runs differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,vocab,dim", EMBED_SHAPES)
@pytest.mark.parametrize("add,offset", [(False, 0), (True, 3)])
def test_embed_grad(dtype, tokens, vocab, dim, add, offset):
    g = gen(tokens * 5 + dim)
    d_out = act(g, tokens, dim, dtype, 0.1)
    ids = torch.randint(-1, vocab, (tokens,), generator=g, device=DEV)
    check_embed_grad(d_out, ids if add else ids.int(), 2.5, add, vocab, dtype, offset, seed=dim)


@pytest.mark.parametrize("tokens", [31, 32, 33, 64, 95, 96, 97, 1000, 2047, 2049, 8191, 8193, 70001])
def test_embed_grad_long_runs(tokens):
    """One number in every token, two halves, a run from and to every phase of a cell."""
    g = gen(tokens)
    dim, vocab = 72, 41
    d_out = act(g, tokens, dim, "f16", 0.1)
    for ids in (torch.full((tokens,), 40), torch.arange(tokens) * 2 // max(tokens, 1),
                (torch.arange(tokens) % 3) * 20, torch.arange(tokens) // 45 % 41):
        check_embed_grad(d_out, ids.to(DEV), 1.0, False, vocab, "f16", pitch=80)


@pytest.mark.parametrize("tokens,vocab", [(65536, 50257), (65537, 300000), (150001, 1000)])
def test_embed_grad_many_tokens(tokens, vocab):
    g = gen(tokens)
    u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * torch.log(torch.tensor(float(vocab)))).long().clamp(1, vocab) - 1
    check_embed_grad(act(g, tokens, 40, "bf16", 0.1), ids, 40.0, False, vocab, "bf16")


@pytest.mark.parametrize("tokens,vocab,dim", [(16000, 700, 801), (13001, 20000, 1607), (21011, 1200, 45), (20001, 333, 130),
                                              (70, 90, 1), (33, 2000, 7), (2049, 5, 9)])
@pytest.mark.parametrize("add,offset,pad", [(False, 0, 0), (False, 1, 0), (False, 7, 3), (True, 2, 0), (True, 5, 0), (True, 0, 7)])
def test_embed_grad_rows_anywhere(tokens, vocab, dim, add, offset, pad):
    """Table rows that start on any element, with ends of every length, in short and long batches."""
    g = gen(tokens + dim + offset)
    u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * torch.log(torch.tensor(float(vocab)))).long().clamp(1, vocab) - 1
    ids[::11] = -1
    check_embed_grad(act(g, tokens, dim, "bf16", 0.1), ids, 0.5, add, vocab, "bf16", offset, pitch=dim + pad, seed=dim)


def test_embed_grad_ids_outside_the_table():
    g = gen(2)
    d_out, table = act(g, 100, 16, "f16"), table_of(g, 10, 16, "f16")
    ids = torch.randint(0, 10, (100,), generator=g, device=DEV)
    ids[::7], ids[3] = -5, 1 << 40
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    run_embed_grad(d_out, ids, 1.0, False, table, bad)
    total, size, count = ref.embed_grad(d_out, ids, 1.0, 10)
    err = (count + 3)[:, None] * ref.E32 * size
    ref.assert_within(table.t, total, ref.U["f16"] * total.abs() + 2 * err + ref.TINY["f16"], "d_table")
    assert int(bad) == 1
    bad.zero_()
    run_embed_grad(d_out, ids.clamp(max=9), 1.0, False, table, bad)
    assert int(bad) == 0
    # nothing but padding: all rows are stored as zero, or left alone
    run_embed_grad(d_out, torch.full_like(ids, -1), 1.0, False, table)
    assert not table.t.any()


def test_embed_gradient_is_the_lookups_transpose():
    """<lookup(E + D) - lookup(E), g> = <D, grad>, by differences of the operator itself
    (values on a coarse grid, so that every operation is exact)."""
    g = gen(8)
    vocab, dim, tokens = 50, 24, 333
    grid = lambda *n: torch.randint(-3, 4, n, generator=g, device=DEV).half() * 0.25  # noqa: E731
    e, d, up = grid(vocab, dim), grid(vocab, dim), grid(tokens, dim)
    ids = torch.randint(-1, vocab, (tokens,), generator=g, device=DEV)
    a, b = torch.empty_like(up), torch.empty_like(up)
    z.zero_embed_lookup(z.mat(e + d), z.ids(ids), 2.0, z.mat(a))
    z.zero_embed_lookup(z.mat(e), z.ids(ids), 2.0, z.mat(b))
    grad = Banded(vocab, dim, torch.float16, pitch=dim)
    run_embed_grad(up, ids, 2.0, False, grad)
    assert float(((a - b).double() * up.double()).sum()) == float((d.double() * grad.t.double()).sum())


# -- weight gradient -------------------------------------------------------------------


def make_ckpt(g, rows, cols, dtype, sigma=1.0, big=8.0):
    x = act(g, rows, cols, dtype, sigma, big)
    q, s = new_act8(rows, cols)
    z.zero_act_pack(z.mat(x), z.act8(q.t, s.t))
    return q.t, s.t


def check_weight_grad(tokens, outs, ins, dtype, gain, add, offset=0, pitch=None, seed=0):
    g = gen(seed + tokens + 3 * outs + 7 * ins)
    t = ref.TYPES[dtype]
    dy = act(g, tokens, outs, dtype, 0.1)
    q, s = make_ckpt(g, tokens, ins, dtype)
    w = (1 + 0.2 * torch.randn(ins + 1, generator=g, device=DEV)).to(t)[1:] if gain else None
    old = torch.randn(outs, ins, generator=g, device=DEV).to(t)
    dw = Banded(outs, ins, t, pitch=pitch or ins, offset=offset, fill=old)
    ws = workspace(z.zero_act_weight_grad_workspace(tokens, outs, ins))
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), w, add, z.mat(dw.t), ws, ws.numel())
    dw64, size = ref.weight_grad(dy, ref.values(q, s), w, old if add else None)
    # products of 16-bit values are exact in fp32; the tensor cores' sums may
    # drop the bits below one part in 2^23 of the running sum at each addition
    err = (tokens + 4) * 2 * ref.E32 * size
    ref.assert_within(dw.t, dw64, ref.U[dtype] * (dw64.abs() + err) + err + ref.TINY[dtype], "dw")
    dw.check("dw")
    again = Banded(outs, ins, t, pitch=pitch or ins, offset=offset, fill=old)
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), w, add, z.mat(again.t), ws, ws.numel())
    assert torch.equal(again.t, dw.t), "two runs differ"


WGRAD_SHAPES = [(1, 1, 1), (1, 16, 16), (2, 300, 200), (63, 128, 128), (64, 256, 128), (65, 129, 257),
                (127, 7, 1601), (100, 1001, 9), (513, 384, 640), (1000, 768, 520), (4100, 136, 264)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,outs,ins", WGRAD_SHAPES)
@pytest.mark.parametrize("gain,add,offset", [(False, False, 0), (True, True, 3)])
def test_weight_grad(dtype, tokens, outs, ins, gain, add, offset):
    check_weight_grad(tokens, outs, ins, dtype, gain, add, offset)


@pytest.mark.parametrize("tokens,outs,ins,pitch", [(2049, 1001, 768, 768), (4096, 1600, 1600, 1608),
                                                   (333, 2600, 2056, 2057)])
def test_weight_grad_larger(tokens, outs, ins, pitch):
    check_weight_grad(tokens, outs, ins, "bf16", True, False, pitch=pitch)
    check_weight_grad(tokens, outs, ins, "f16", False, True, pitch=pitch)


@pytest.mark.parametrize("tokens,outs,ins,pitch,offset", [
    (70, 5001, 2100, 2104, 0), (5, 4096, 2560, 2560, 8), (130, 2600, 2056, 2056, 0), (1030, 4343, 2071, 2080, 16),
    (1, 9000, 544, 544, 2)])
@pytest.mark.parametrize("add", [False, True])
def test_weight_grad_more_tiles_than_pairs(tokens, outs, ins, pitch, offset, add):
    """A pair of CTAs takes several tiles, and writes one while it multiplies the next."""
    check_weight_grad(tokens, outs, ins, "f16", True, add, offset, pitch)


@pytest.mark.parametrize("dtype", DTYPES)
def test_weight_grad_of_lost_blocks_and_infinities(dtype):
    """A NaN block poisons its 32 columns, an infinite gradient its row; nothing else."""
    g = gen(9)
    tokens, outs, ins = 70, 40, 96
    dy = act(g, tokens, outs, dtype, 0.1)
    x = act(g, tokens, ins, dtype)
    x[13, 33] = float("inf")
    dy[20, 7] = float("inf")
    q, s = z.act8_empty(tokens, ins)
    z.zero_act_pack(z.mat(x), z.act8(q, s))
    dw = torch.empty(outs, ins, dtype=ref.TYPES[dtype], device=DEV)
    ws = workspace(z.zero_act_weight_grad_workspace(tokens, outs, ins))
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), None, False, z.mat(dw), ws, ws.numel())
    bad = ~torch.isfinite(dw)
    want = torch.zeros_like(bad)
    want[:, 32:64] = True
    want[7] = True
    assert torch.equal(bad, want)


def test_weight_grad_is_linear_in_the_weight():
    """<X D^T, dy> = <D, dw> for any D, with the layer's own product in 64 bits."""
    g = gen(21)
    tokens, outs, ins = 200, 72, 88
    dy = torch.randint(-2, 3, (tokens, outs), generator=g, device=DEV).half()
    x = torch.randint(-3, 4, (tokens, ins), generator=g, device=DEV).half()
    q, s = z.act8_empty(tokens, ins)
    z.zero_act_pack(z.mat(x), z.act8(q, s))
    dw = torch.empty(outs, ins, dtype=torch.float16, device=DEV)
    ws = workspace(z.zero_act_weight_grad_workspace(tokens, outs, ins))
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), None, False, z.mat(dw), ws, ws.numel())
    d = torch.randn(outs, ins, generator=g, device=DEV).double()
    y = lambda w: x.double() @ w.t()  # noqa: E731
    num = float(((y(d) - y(-d)) / 2 * dy.double()).sum())
    assert float((dw.double() * d).sum()) == pytest.approx(num, rel=1e-10)


# -- all of them -------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
def test_nothing_to_sum(dtype):
    """No tokens: no activation is written, a stored gradient is zero, an added one stays."""
    t = ref.TYPES[dtype]
    none = torch.empty(0, 64, dtype=t, device=DEV)
    q, s = z.act8_empty(0, 64)
    c, no_ids = z.act8(q, s), z.ids(torch.empty(0, dtype=torch.int64, device=DEV))
    rstd = torch.empty(0, device=DEV)
    one = torch.ones(40, 64, dtype=t, device=DEV)
    table, dw, dg = one.clone(), one.clone(), one[0].clone()
    ws = workspace(1 << 20)
    for add in (True, False):
        z.zero_embed_lookup(z.mat(one), no_ids, 1.0, z.mat(none))
        z.zero_embed_grad(z.mat(none), no_ids, 1.0, add, z.mat(table), ws, ws.numel())
        z.zero_norm_forward(z.mat(none), None, None, 1e-5, None, z.mat(torch.empty_like(none)), rstd, c)
        z.zero_norm_backward(z.mat(none), c, rstd, None, None, z.mat(none), dg, add, ws, ws.numel())
        z.zero_act_pack(z.mat(none), c)
        z.zero_act_unpack(c, z.mat(none))
        z.zero_act_weight_grad(z.mat(torch.empty(0, 40, dtype=t, device=DEV)), c, None, add, z.mat(dw), ws,
                               ws.numel())
        want = 1.0 if add else 0.0
        for got in (table, dw, dg):
            assert bool((got == want).all())


def test_column_slices_of_one_buffer():
    """Inputs and outputs that interleave in one buffer without sharing an element."""
    g = gen(31)
    rows, cols = 50, 64
    both = torch.randn(rows, 2 * cols, generator=g, device=DEV).half()
    x = both[:, :cols].clone()
    z.zero_norm_forward(z.mat(both[:, :cols]), None, None, 1e-5, None, z.mat(both[:, cols:]))
    y = torch.empty_like(x)
    z.zero_norm_forward(z.mat(x), None, None, 1e-5, None, z.mat(y))
    assert torch.equal(both[:, :cols], x) and torch.equal(both[:, cols:], y)


def test_other_stream_and_graph():
    """On a stream of the caller's, and captured in a CUDA graph: the same bits."""
    g = gen(30)
    tokens, dim, outs, vocab = 700, 320, 200, 1000
    table = table_of(g, vocab, dim, "bf16").t
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).bfloat16()
    dyo, dy = act(g, tokens, outs, "bf16"), act(g, tokens, dim, "bf16")
    x = torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    rstd, dg = torch.empty(tokens, device=DEV), torch.empty_like(w)
    q, s = z.act8_empty(tokens, dim)
    dw = torch.empty(outs, dim, dtype=torch.bfloat16, device=DEV)
    dt = torch.empty(vocab, dim, dtype=torch.bfloat16, device=DEV)
    ws = [workspace(z.zero_norm_backward_workspace(tokens, dim)),
          workspace(z.zero_act_weight_grad_workspace(tokens, outs, dim)),
          workspace(z.zero_embed_grad_workspace(tokens, vocab, dim))]
    c = z.act8(q, s)

    def chain(stream):
        z.zero_embed_lookup(z.mat(table), z.ids(ids), 2.0, z.mat(x), None, stream)
        z.zero_norm_forward(z.mat(x), None, w, 1e-5, None, z.mat(y), rstd, c, stream)
        z.zero_act_weight_grad(z.mat(dyo), c, w, False, z.mat(dw), ws[1], ws[1].numel(), stream)
        z.zero_norm_backward(z.mat(dy), c, rstd, w, None, z.mat(dx), dg, False, ws[0], ws[0].numel(), stream)
        z.zero_embed_grad(z.mat(dx), z.ids(ids), 2.0, False, z.mat(dt), ws[2], ws[2].numel(), None, stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (x, y, rstd, q, s, dw, dx, dg, dt)]

    chain(None)
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for out in (x, y, dx, dw, dt):
        out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    chain(side)
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        chain(side)
    for out in (x, y, dx, dw, dt):
        out.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(results(), want))


def test_calls_in_a_row_share_buffers(monkeypatch):
    """Calls issued back to back on one stream, alternating inputs and sharing their
    output and workspace, each give what they give alone: with dependent launches,
    whose kernels start while the call before still runs, and with plain ones."""
    g = gen(50)
    vocab, dim, tokens, outs = 5000, 264, 3000, 520
    sets = []
    for k in range(3):
        ids = torch.randint(0, vocab // (k + 1), (tokens - 500 * k,), generator=g, device=DEV)
        n = ids.numel()
        x = act(g, n, dim, "bf16", 1.0, 5.0)
        sets.append(dict(ids=ids, x=x, dy=act(g, n, dim, "bf16"), dyo=act(g, n, outs, "bf16")))
    table, dw = (torch.empty(r, dim, dtype=torch.bfloat16, device=DEV) for r in (vocab, outs))
    dg = torch.empty(dim, dtype=torch.bfloat16, device=DEV)
    rstd = torch.empty(tokens, device=DEV)
    store = torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV)
    q, s = z.act8_empty(tokens, dim)
    ws = workspace(max(z.zero_embed_grad_workspace(tokens, vocab, dim),
                       z.zero_act_weight_grad_workspace(tokens, outs, dim),
                       z.zero_norm_backward_workspace(tokens, dim)))

    def call(c, copy):
        n = c["ids"].numel()
        k, dx = z.act8(q[:n], s[:n]), store[:n]
        z.zero_norm_forward(z.mat(c["x"]), None, None, 1e-5, None, z.mat(dx), rstd, k)
        z.zero_act_weight_grad(z.mat(c["dyo"]), k, None, False, z.mat(dw), ws, ws.numel())
        z.zero_norm_backward(z.mat(c["dy"]), k, rstd, None, None, z.mat(dx), dg, False, ws, ws.numel())
        z.zero_embed_grad(z.mat(dx), z.ids(c["ids"]), 1.0, False, z.mat(table), ws, ws.numel())
        return [t.clone() for t in (table, dw, dg)] if copy else None

    alone = []
    for c in sets:
        torch.cuda.synchronize()
        alone.append(call(c, True))
        torch.cuda.synchronize()
    for pdl in ("1", "0"):
        monkeypatch.setenv("ZERO_PDL", pdl)
        for last in range(3):
            for i in range(9):
                call(sets[(last + 1 + i) % 3], False)
            assert (last + 9) % 3 == last
            got = call(sets[last], True)
            assert all(torch.equal(a, b) for a, b in zip(got, alone[last]))


def test_rows_far_apart():
    """Rows 4 GB apart: element offsets past 2^32 in every operator."""
    far, rows, cols = 1 << 31, 4, 40
    store = torch.empty(rows * far, dtype=torch.float16, device=DEV)       # 16 GB
    x = torch.as_strided(store, (rows, cols), (far, 1), 0)
    out = torch.as_strided(store, (rows, cols), (far, 1), 64)
    g = gen(40)
    x.copy_(torch.randn(rows, cols, generator=g, device=DEV))
    near = x.contiguous()
    qs = torch.zeros(rows * far, dtype=torch.int8, device=DEV)             # 8 GB
    q = torch.as_strided(qs, (rows, cols), (far, 1), 0)
    s = torch.empty(rows, 2, dtype=torch.uint8, device=DEV)
    z.zero_act_pack(z.mat(x), z.act8(q, s))
    q2, s2 = z.act8_empty(rows, cols)
    z.zero_act_pack(z.mat(near), z.act8(q2, s2))
    assert torch.equal(q, q2) and torch.equal(s, s2)
    z.zero_act_unpack(z.act8(q, s), z.mat(out))
    assert torch.equal(out.cpu().double(), ref.values(q2.cpu(), s2.cpu()))
    y = torch.empty_like(near)
    rstd, r2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    z.zero_norm_forward(z.mat(x), None, None, 1e-5, None, z.mat(out), rstd, z.act8(q, s))
    z.zero_norm_forward(z.mat(near), None, None, 1e-5, None, z.mat(y), r2, z.act8(q2, s2))
    assert torch.equal(out, y) and torch.equal(rstd, r2) and torch.equal(q, q2)
    ws = workspace(1 << 20)
    dg, dg2 = torch.empty(cols, dtype=torch.float16, device=DEV), torch.empty(cols, dtype=torch.float16, device=DEV)
    z.zero_norm_backward(z.mat(x), z.act8(q, s), rstd, None, None, z.mat(out), dg, False, ws, ws.numel())
    z.zero_norm_backward(z.mat(near), z.act8(q2, s2), r2, None, None, z.mat(y), dg2, False, ws, ws.numel())
    assert torch.equal(out, y) and torch.equal(dg, dg2)
    n = z.zero_act_weight_grad_workspace(rows, cols, cols)
    ws = workspace(n)
    dw = torch.as_strided(store, (cols // 10, cols), (far, 1), 128)
    dw2 = torch.empty(cols // 10, cols, dtype=torch.float16, device=DEV)
    z.zero_act_weight_grad(z.mat(x[:, :4]), z.act8(q, s), None, False, z.mat(dw), ws, n)
    z.zero_act_weight_grad(z.mat(near[:, :4]), z.act8(q2, s2), None, False, z.mat(dw2), ws, n)
    assert torch.equal(dw, dw2)
    ids = torch.tensor([3, 0, 2, 3], device=DEV)
    z.zero_embed_lookup(z.mat(x), z.ids(ids), 1.0, z.mat(out))
    assert torch.equal(out, near[ids])
    n = z.zero_embed_grad_workspace(rows, rows, cols)
    ws = workspace(n)
    z.zero_embed_grad(z.mat(x), z.ids(ids), 1.0, False, z.mat(out), ws, n)
    total, _, _ = ref.embed_grad(near, ids, 1.0, rows)
    ref.assert_within(out, total, (ref.U["f16"] + 2 * ref.E32) * total.abs() + ref.TINY["f16"], "d_table")
