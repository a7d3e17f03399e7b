"""Every instance of the training operators' kernels, at sizes that choose it
(train_rule): rows of every width that a model has, several turns of a CTA, each
layout of the table gradient; checkpoints of the other 16-bit type; and the
sizes of a training micro-batch."""
import itertools

import pytest
import torch

import test_gpu_train_ops as ops
import train_ref as ref
import train_rule as rule
import zero_sharded_optimizer_02_gb300 as z

DEV = "cuda"
DTYPES = ["f16", "bf16"]

NORM_SHAPES = [(5001, 160), (4001, 512), (4001, 768), (4001, 1000), (4001, 1024), (1300, 4096), (1000, 5000),
               (1000, 5120), (1000, 8192), (3, 8192), (700, 9000), (320, 32768)]
# tokens, vocabulary, columns
TABLE_SHAPES = [(300, 500, 40), (7400, 900, 1608), (16000, 2000, 768), (20100, 700, 24)]


# -- on the CPU: the sizes choose every instance -----------------------------------------


def test_rules_are_the_librarys():
    """Where a workspace's size shows the choice, it is the one written again here."""
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    for rows, cols in itertools.product([1, 3, 200, 607, 608, 609, 5000, 20000],
                                        [1, 8, 33, 504, 505, 512, 1000, 1016, 1017, 1024, 4096, 4097, 8192, 8200, 32768]):
        assert z.zero_norm_backward_workspace(rows, cols) == rule.norm_workspace(rows, cols), (rows, cols)
    for tokens, dim in itertools.product([1, 300, 7296, 7297, 20000, 20001, 65536], [1, 24, 40, 768, 1601, 1608, 2048, 2056]):
        assert z.zero_embed_grad_workspace(tokens, 1000, dim) == rule.table_workspace(tokens, dim), (tokens, dim)


def test_sizes_choose_every_instance():
    every = {(1, False, False), (2, False, True), (2, False, False), (4, False, True), (4, False, False),
             (4, True, False)}
    for backward in (False, True):
        chosen = [rule.norm(r, c, backward) for r, c in NORM_SHAPES]
        assert {c[0] for c in chosen} == every
        assert {c[0] for c in chosen if c[2]} == every, "each with CTAs that take several turns"
        assert {c[0] for c in chosen if c[1] > 1} >= {(1, False, False), (2, False, True), (2, False, False)}
    assert {rule.table_layout(t, d) for t, _, d in TABLE_SHAPES} == {"few", "some", "many"}


# -- on the GPU ------------------------------------------------------------------------------


@pytest.fixture(scope="module")
def built():
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


gpu = [pytest.mark.gpu, pytest.mark.usefixtures("built")]


def on_gpu(fn):
    for m in gpu:
        fn = m(fn)
    return fn


@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_forward(dtype, rows, cols):
    ops.test_norm_forward(dtype, rows, cols, True, True)


@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("residual,gain,add", [(True, True, False), (False, True, True)])
def test_norm_backward(dtype, rows, cols, residual, gain, add):
    ops.test_norm_backward(dtype, rows, cols, residual, gain, add)


@on_gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,vocab,dim", TABLE_SHAPES)
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("offset", [0, 3])
def test_embed_grad(dtype, tokens, vocab, dim, add, offset):
    g = ops.gen(tokens + dim)
    u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * torch.log(torch.tensor(float(vocab)))).long().clamp(1, vocab) - 1
    ids[::13] = -1
    ops.check_embed_grad(ops.act(g, tokens, dim, dtype, 0.1), ids, 2.0, add, vocab, dtype, offset, seed=dim)


def weight_grad(dy, q, s, outs, ins):
    dw = torch.empty(outs, ins, dtype=dy.dtype, device=DEV)
    n = z.zero_act_weight_grad_workspace(dy.shape[0], outs, ins)
    ws = ops.workspace(n)
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), None, False, z.mat(dw), ws, n)
    return dw


@on_gpu
def test_weight_grad_of_a_bfloat16_checkpoint_in_binary16():
    """Its values are rounded to binary16 once: subnormals where steps are under 2^-24 or
    2^-14 apart, infinities past 65,504; a converting path of its own (steps that binary16
    does not hold)."""
    g = ops.gen(61)
    tokens, outs, ins = 200, 72, 160
    x = torch.randn(tokens, ins, generator=g, device=DEV)
    x[:, :32] *= 2.0 ** -18        # steps of about 2^-23, values down to below binary16's least
    x[:, 32:64] *= 2.0 ** -22
    x[:, 64:96] *= 2.0 ** 9        # steps of about 2^4
    x[:, 128:] = x[:, 128:].abs() * 2.0 ** 22 + 2.0 ** 20      # steps of about 2^17: infinite in binary16
    x = x.bfloat16()
    q, s = z.act8_empty(tokens, ins)
    z.zero_act_pack(z.mat(x), z.act8(q, s))
    assert int(s[:, 1].min()) < 127 - 24 and int(s[:, 4].min()) > 127 + 15 and int(s[:, 2].max()) < 142
    dy = (torch.rand(tokens, outs, generator=g, device=DEV) + 0.25).half()
    kept = ref.values(q, s).to(torch.float16).double()
    assert bool(torch.isinf(kept[:, 128:]).all()) and bool(torch.isfinite(kept[:, :128]).all())
    dw = weight_grad(dy, q, s, outs, ins)
    want, size = ref.weight_grad(dy, kept[:, :128], None)
    err = (tokens + 4) * 2 * ref.E32 * size
    assert float(want.abs().max()) < 65504
    ref.assert_within(dw[:, :128], want, ref.U["f16"] * (want.abs() + err) + err + ref.TINY["f16"], "dw")
    assert bool((dw[:, 128:] == float("inf")).all())


@on_gpu
def test_weight_grad_of_a_binary16_checkpoint_in_bfloat16():
    """Whole numbers of 7 bits times 2^-24 to 2^9 are exact in bfloat16."""
    g = ops.gen(62)
    tokens, outs, ins = 300, 40, 96
    x = torch.randn(tokens, ins, generator=g, device=DEV)
    x[:, :32] *= 2.0 ** -18
    x[:, 32:64] *= 2.0 ** 13
    q, s = z.act8_empty(tokens, ins)
    z.zero_act_pack(z.mat(x.half()), z.act8(q, s))
    dy = (torch.randn(tokens, outs, generator=g, device=DEV)).bfloat16()
    dw = weight_grad(dy, q, s, outs, ins)
    want, size = ref.weight_grad(dy, ref.values(q, s), None)
    err = (tokens + 4) * 2 * ref.E32 * size
    ref.assert_within(dw, want, ref.U["bf16"] * (want.abs() + err) + err, "dw")


@on_gpu
def test_norm_of_a_training_micro_batch():
    """16,384 rows of 4,096, forward and backward (which is run twice: the same bits)."""
    ops.test_norm_forward("bf16", 16384, 4096, True, True)
    ops.test_norm_backward("bf16", 16384, 4096, True, True, False)


@on_gpu
def test_weight_grad_of_a_training_micro_batch():
    """16,384 tokens, 4,096 -> 16,384: ten runs give the same bits, and a sample of rows and
    columns is within the bound."""
    tokens, outs, ins = 16384, 16384, 4096
    g = ops.gen(63)
    dy = ops.act(g, tokens, outs, "bf16", 1e-3)
    q, s = ops.make_ckpt(g, tokens, ins, "bf16")
    first = weight_grad(dy, q, s, outs, ins)
    for _ in range(9):
        assert torch.equal(weight_grad(dy, q, s, outs, ins), first)
    rows = torch.randperm(outs, generator=g, device=DEV)[:200]
    cols = torch.randperm(ins, generator=g, device=DEV)[:100]
    want, size = ref.weight_grad(dy[:, rows], ref.values(q, s)[:, cols], None)
    err = (tokens + 4) * 2 * ref.E32 * size
    ref.assert_within(first[rows][:, cols], want, ref.U["bf16"] * (want.abs() + err) + err, "dw")
