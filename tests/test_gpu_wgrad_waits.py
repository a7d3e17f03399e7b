"""The weight gradient's kernel when a wait runs out: what it has not finished
is NaN, and every element that is not NaN is right.

Its waits are on its own copies and products, which always arrive, so the
kernel is launched here with arguments of the test's (tests/c/wgrad_waits.cu):
copies of half a step's tokens, whose missing bytes nothing brings, with a wait
of 20 ms; or whole copies with a wait far shorter than a tile takes.  Every
access stays inside its buffers, every wait ends, and the CUDA context stays
usable."""
import ctypes as C
import os
import subprocess
import time

import pytest
import torch

import zero_sharded_optimizer_02_gb300 as z
from test_gpu_train_ops import act, gen, make_ckpt, workspace

pytestmark = pytest.mark.gpu

DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))
SHORT_WAIT_NS = 20_000_000


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    so = str(tmp_path_factory.mktemp("waits") / "libwaits.so")
    subprocess.check_call([build._nvcc(), "-O3", "-std=c++17", *build.ARCH, "-shared", "-Xcompiler", "-fPIC",
                           "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(HERE, "c", "wgrad_waits.cu"),
                           os.path.join(build.CSRC, "zero_train_host.cpp"), "-o", so])
    fn = C.CDLL(so).wgrad_waits
    fn.argtypes = [C.POINTER(z.Mat), C.POINTER(z.Act8), C.c_uint32, C.POINTER(z.Mat), C.c_void_p, C.c_uint64,
                   C.c_uint64, C.c_uint32, C.c_uint32, C.c_uint32]
    fn.restype = C.c_int

    def call(dy, q, s, add, dw, wait_ns, short_dy=False, short_q=False, one_pair=False):
        n = z.zero_act_weight_grad_workspace(dy.shape[0], dy.shape[1], q.shape[1])
        ws = workspace(n)
        torch.cuda.synchronize()
        assert fn(z.mat(dy), z.act8(q, s), int(add), z.mat(dw), ws.data_ptr(), n, wait_ns, short_dy, short_q,
                  one_pair) == 0
        torch.cuda.synchronize()   # no error: the context stays usable
        return dw

    return call


def problem(tokens, outs, ins, dtype):
    g = gen(tokens + outs)
    dy = act(g, tokens, outs, dtype, 0.1)
    return (dy, *make_ckpt(g, tokens, ins, dtype))


def right(dy, q, s, add, old):
    """The entry point's result."""
    dw = old.clone()
    n = z.zero_act_weight_grad_workspace(dy.shape[0], *dw.shape)
    ws = workspace(n)
    z.zero_act_weight_grad(z.mat(dy), z.act8(q, s), None, add, z.mat(dw), ws, n)
    return dw


@pytest.mark.parametrize("short", ["dy", "checkpoint"])
def test_a_wait_that_runs_out_ends_the_call_soon(run, short):
    """20 ms for the waits and 1 s for all copies that may still be under way, not 4 s for each."""
    dy, q, s = problem(450, 1024, 1000, "bf16")
    dw = torch.ones(1024, 1000, dtype=torch.bfloat16, device=DEV)
    run(dy, q, s, False, dw, 10 ** 9)          # loads the kernels
    want = dw.clone()
    t0 = time.monotonic()
    run(dy, q, s, False, dw, SHORT_WAIT_NS, short_dy=short == "dy", short_q=short == "checkpoint")
    assert time.monotonic() - t0 < 3.0
    assert bool(torch.isnan(dw).all())
    assert torch.equal(right(dy, q, s, False, dw), want)   # an ordinary call afterwards


def test_a_wait_that_runs_out_under_products(run):
    """Nothing is missing, but the epilogue's waits, which look at the clock every 64 tries,
    run out on tiles of 16,000 steps (5 ms), while products are issued.  The call ends, and
    an undisturbed one behind it gives what it gave before."""
    dy, q, s = problem(1_024_000, 1024, 512, "bf16")
    old = torch.randn(1024, 512, generator=gen(1), device=DEV).bfloat16()
    whole = run(dy, q, s, True, old.clone(), 10 ** 9, one_pair=True)
    assert bool(torch.isfinite(whole).all())
    for wait_ns in (0, 100_000):
        lost = run(dy, q, s, True, old.clone(), wait_ns, one_pair=True)
        assert bool(torch.isnan(lost).any())
        assert torch.equal(run(dy, q, s, True, old.clone(), 10 ** 9, one_pair=True), whole)


@pytest.mark.parametrize("short", ["dy", "checkpoint"])
@pytest.mark.parametrize("tokens,add,pad", [(64, False, 0), (64, True, 3), (450, False, 0)])
def test_nothing_unfinished_looks_finished(run, short, tokens, add, pad):
    """Nothing can be multiplied from the first step on: all of dw is NaN, also the third and
    later tiles of a pair, whose barrier's last phase has the parity that their waits look
    for; as for tiles stored at once (16 tiles, one pair), so for those cut along the tokens."""
    outs, ins = 1024, 1000
    dy, q, s = problem(tokens, outs, ins, "bf16")
    dw = torch.ones(outs, ins + pad, dtype=torch.bfloat16, device=DEV)[:, :ins]
    run(dy, q, s, add, dw, SHORT_WAIT_NS, short_dy=short == "dy", short_q=short == "checkpoint",
        one_pair=tokens == 64)
    assert bool(torch.isnan(dw).all()), f"{int((~torch.isnan(dw)).sum())} elements look finished"


def test_whatever_is_finished_is_right(run):
    """Waits that run out while products are issued, on tiles of 5 ms: elements are NaN or those
    of an undisturbed run."""
    dy, q, s = problem(1_024_000, 1024, 512, "bf16")
    old = torch.randn(1024, 512, generator=gen(1), device=DEV).bfloat16()
    whole = run(dy, q, s, True, old.clone(), 10 ** 9, one_pair=True)
    for wait_ns in (0, 100_000, 1_000_000, 4_000_000):
        dw = run(dy, q, s, True, old.clone(), wait_ns, one_pair=True)
        lost = torch.isnan(dw)
        assert wait_ns > 1_000_000 or bool(lost.any())
        assert torch.equal(dw[~lost], whole[~lost]), f"wait of {wait_ns} ns"
