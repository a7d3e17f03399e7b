"""The losses' kernel when a wait between the CTAs of a row runs out: the loss and
the gradient of the rows not finished are NaN, and the call ends.

The CTAs' sums always arrive, so the kernel is launched here with arguments of
the test's (tests/c/loss_waits.cu): it waits for 8 bytes a row more than they
send.  Every access stays inside its buffers, the wait ends after 20 ms, and the
CUDA context stays usable."""
import ctypes as C
import os
import subprocess
import time

import pytest
import torch

import zero_sharded_optimizer_02_gb300 as z
from test_gpu_loss_ops import batch, grad_of

pytestmark = pytest.mark.gpu

DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))
WAIT_NS = 20_000_000


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    so = str(tmp_path_factory.mktemp("waits") / "liblosswaits.so")
    subprocess.check_call([build._nvcc(), "-O3", "-std=c++17", *build.ARCH, "-shared", "-Xcompiler", "-fPIC",
                           "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(HERE, "c", "loss_waits.cu"),
                           os.path.join(build.CSRC, "zero_train_host.cpp"), "-o", so])
    fn = C.CDLL(so).loss_waits
    fn.argtypes = [C.POINTER(z.Mat), C.POINTER(z.Ids), C.c_void_p, C.POINTER(z.Mat), C.c_uint64, C.c_uint32]
    fn.restype = C.c_int

    def call(x, targets, missing):
        loss, d = torch.full((x.shape[0],), 3.0, device=DEV), grad_of(x)
        torch.cuda.synchronize()
        start = time.monotonic()
        assert fn(z.mat(x), z.ids(targets), loss.data_ptr(), z.mat(d.t), WAIT_NS, missing) == 0
        torch.cuda.synchronize()   # no error: the context stays usable
        d.check()
        return loss, d.t, time.monotonic() - start

    return call


@pytest.mark.parametrize("rows", [1, 8, 45])
def test_sums_that_never_come(run, rows):
    _, x, targets = batch(rows, rows, 9001, "bf16", pad=0.2)
    gone = targets < 0
    loss, d, _ = run(x, targets, 0)            # loads the kernel; nothing is missing
    want, d_want = torch.empty(rows, device=DEV), grad_of(x)
    z.zero_distill_loss(z.mat(x), None, None, 1.0, 0.0, z.ids(targets), 1.0, None, 1.0, want, z.mat(d_want.t))
    assert torch.allclose(loss, want, rtol=1e-5, atol=1e-6)
    # each of 8 clusters waits once; the rows behind that have no further limit to wait for
    loss, d, seconds = run(x, targets, 8)
    assert seconds < 1.0
    assert bool(torch.isnan(loss[~gone]).all()) and bool((loss[gone] == 0).all())
    assert bool(torch.isnan(d[~gone]).all()) and bool((d[gone] == 0).all())
    # and the library's own call gives what it gave before
    again, d_again = torch.empty(rows, device=DEV), grad_of(x)
    z.zero_distill_loss(z.mat(x), None, None, 1.0, 0.0, z.ids(targets), 1.0, None, 1.0, again, z.mat(d_again.t))
    assert torch.equal(again, want) and torch.equal(d_again.t, d_want.t)
