"""Refusals of the training operators, without a GPU: every invalid argument is
reported on the host and nothing is launched.  The addresses are never
dereferenced: each call fails validation before any CUDA call, or has nothing
to do."""
import ctypes as C

import pytest
import torch

import train_ref as ref

A = 1 << 20          # a 16-byte aligned address
STEP = 1 << 30       # further apart than any buffer below


@pytest.fixture(scope="module")
def z():
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    import zero_sharded_optimizer_02_gb300 as z
    return z


def mat(z, at, rows, cols, pitch=None, dtype=None):
    return z.Mat(at, rows, cols, -(-cols // 8) * 8 if pitch is None else pitch,
                 z.ZERO_F16 if dtype is None else dtype)


def ckpt(z, at, rows, cols, q_pitch=None, scale_pitch=None, scale_at=None):
    nb = -(-cols // 32)
    return z.Act8(at, at + STEP // 2 if scale_at is None else scale_at, rows, cols,
                  -(-cols // 16) * 16 if q_pitch is None else q_pitch,
                  nb if scale_pitch is None else scale_pitch)


def refused(z, status, fn, *args):
    with pytest.raises(z.ZeroError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def at(k):
    return A + k * STEP


def lookup_args(z, **kw):
    a = dict(table=mat(z, at(1), 100, 64), ids=z.Ids(at(2), 10, 8), scale=1.0,
             out=mat(z, at(3), 10, 64), bad=at(4))
    a.update(kw)
    return list(a.values())


def egrad_args(z, **kw):
    a = dict(d_out=mat(z, at(3), 10, 64), ids=z.Ids(at(2), 10, 8), scale=1.0, add=False,
             table=mat(z, at(1), 100, 64), ws=at(5), n=1 << 24, bad=at(4))
    a.update(kw)
    return list(a.values())


def forward_args(z, **kw):
    a = dict(x=mat(z, at(1), 10, 64), res=mat(z, at(2), 10, 64), gain=at(3), eps=1e-5,
             h=mat(z, at(4), 10, 64), y=mat(z, at(5), 10, 64), rstd=at(6), c=ckpt(z, at(7), 10, 64))
    a.update(kw)
    return list(a.values())


def backward_args(z, **kw):
    a = dict(dy=mat(z, at(1), 10, 64), c=ckpt(z, at(2), 10, 64), rstd=at(3), gain=at(4),
             dres=mat(z, at(5), 10, 64), dx=mat(z, at(6), 10, 64), dg=at(7), add=False, ws=at(8),
             n=1 << 24)
    a.update(kw)
    return list(a.values())


def wgrad_args(z, **kw):
    a = dict(dy=mat(z, at(1), 10, 40), c=ckpt(z, at(2), 10, 64), gain=at(3), add=False,
             dw=mat(z, at(4), 40, 64), ws=at(5), n=1 << 40)
    a.update(kw)
    return list(a.values())


BAD_MATS = [  # (what differs from a good activation matrix, status)
    (dict(at=A + 2), 2), (dict(pitch=65), 2), (dict(pitch=56), 1), (dict(dtype=2), 1),
    (dict(dtype=-1), 1), (dict(at=None), 1), (dict(pitch=1 << 57), 1)]


def _variant(z, k, rows, cols, d):
    d = dict(d)
    d.setdefault("at", at(k))
    return mat(z, d.pop("at"), rows, cols, **d)


def test_activation_matrices(z):
    for d, status in BAD_MATS:
        refused(z, status, z.zero_embed_lookup, *lookup_args(z, out=_variant(z, 3, 10, 64, d)))
        refused(z, status, z.zero_embed_grad, *egrad_args(z, d_out=_variant(z, 3, 10, 64, d)))
        for k, name in ((1, "x"), (2, "res"), (4, "h"), (5, "y")):
            refused(z, status, z.zero_norm_forward, *forward_args(z, **{name: _variant(z, k, 10, 64, d)}))
        for k, name in ((1, "dy"), (5, "dres"), (6, "dx")):
            refused(z, status, z.zero_norm_backward, *backward_args(z, **{name: _variant(z, k, 10, 64, d)}))
        refused(z, status, z.zero_act_pack, _variant(z, 1, 10, 64, d), ckpt(z, at(2), 10, 64))
        refused(z, status, z.zero_act_unpack, ckpt(z, at(2), 10, 64), _variant(z, 1, 10, 64, d))
        refused(z, status, z.zero_act_weight_grad, *wgrad_args(z, dy=_variant(z, 1, 10, 40, dict(d, pitch=d["pitch"] - 24) if d.get("pitch", 0) in (56, 65) else d)))


def test_parameter_matrices_need_two_byte_alignment_only(z):
    for fn, args, name, rows in ((z.zero_embed_lookup, lookup_args, "table", 100),
                                 (z.zero_embed_grad, egrad_args, "table", 100),
                                 (z.zero_act_weight_grad, wgrad_args, "dw", 40)):
        refused(z, 2, fn, *args(z, **{name: mat(z, A + 1, rows, 64)}))
        refused(z, 1, fn, *args(z, **{name: mat(z, at(1), rows, 64, pitch=63)}))
        refused(z, 1, fn, *args(z, **{name: mat(z, None, rows, 64)}))


def test_checkpoints(z):
    for bad, status in ((dict(q_pitch=72), 2), (dict(q_pitch=48), 1), (dict(scale_pitch=1), 1),
                        (dict(at=A + 8), 2), (dict(scale_at=None, at=None), 1)):
        d = dict(bad)
        where = d.pop("at", at(7))
        c = z.Act8(None, None, 10, 64, 64, 2) if where is None else ckpt(z, where, 10, 64, **d)
        refused(z, status, z.zero_norm_forward, *forward_args(z, c=c))
        refused(z, status, z.zero_norm_backward, *backward_args(z, c=c))
        refused(z, status, z.zero_act_pack, mat(z, at(1), 10, 64), c)
        refused(z, status, z.zero_act_unpack, c, mat(z, at(1), 10, 64))
        refused(z, status, z.zero_act_weight_grad, *wgrad_args(z, c=c))


def test_shapes_that_disagree(z):
    other = [(9, 64), (10, 63)]
    for r, c in other:
        refused(z, 1, z.zero_embed_lookup, *lookup_args(z, out=mat(z, at(3), r, c)))
        refused(z, 1, z.zero_embed_grad, *egrad_args(z, d_out=mat(z, at(3), r, c)))
        for name in ("res", "h", "y"):
            refused(z, 1, z.zero_norm_forward, *forward_args(z, **{name: mat(z, at(9), r, c)}))
        refused(z, 1, z.zero_norm_forward, *forward_args(z, c=ckpt(z, at(9), r, c)))
        for name in ("dres", "dx"):
            refused(z, 1, z.zero_norm_backward, *backward_args(z, **{name: mat(z, at(9), r, c)}))
        refused(z, 1, z.zero_norm_backward, *backward_args(z, c=ckpt(z, at(9), r, c)))
        refused(z, 1, z.zero_act_pack, mat(z, at(1), 10, 64), ckpt(z, at(2), r, c))
        refused(z, 1, z.zero_act_unpack, ckpt(z, at(2), r, c), mat(z, at(1), 10, 64))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=mat(z, at(4), 41, 64)))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=mat(z, at(4), 40, 63)))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, c=ckpt(z, at(2), 11, 64)))
    # types that disagree
    refused(z, 1, z.zero_embed_lookup, *lookup_args(z, out=mat(z, at(3), 10, 64, dtype=1)))
    refused(z, 1, z.zero_embed_grad, *egrad_args(z, table=mat(z, at(1), 100, 64, dtype=1)))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, y=mat(z, at(5), 10, 64, dtype=1)))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, dx=mat(z, at(6), 10, 64, dtype=1)))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=mat(z, at(4), 40, 64, dtype=1)))


def test_scalars_flags_and_small_pointers(z):
    for s in (float("nan"), float("inf")):
        refused(z, 1, z.zero_embed_lookup, *lookup_args(z, scale=s))
        refused(z, 1, z.zero_embed_grad, *egrad_args(z, scale=s))
    for e in (0.0, -1e-5, float("nan"), float("inf")):
        refused(z, 1, z.zero_norm_forward, *forward_args(z, eps=e))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, h=None, y=None, rstd=None, c=None))
    for fn, args in ((z.zero_embed_grad, egrad_args), (z.zero_norm_backward, backward_args),
                     (z.zero_act_weight_grad, wgrad_args)):
        refused(z, 1, fn, *args(z, add=2))
    for fn, args in ((z.zero_embed_lookup, lookup_args), (z.zero_embed_grad, egrad_args)):
        refused(z, 2, fn, *args(z, bad=at(4) + 2))
        refused(z, 2, fn, *args(z, ids=z.Ids(at(2) + 4, 10, 8)))
        refused(z, 1, fn, *args(z, ids=z.Ids(at(2), 10, 2)))
        refused(z, 1, fn, *args(z, ids=z.Ids(None, 10, 8)))
        refused(z, 5, fn, *args(z, ids=z.Ids(at(2), 1 << 31, 8)))
    refused(z, 2, z.zero_norm_forward, *forward_args(z, gain=at(3) + 1))
    refused(z, 2, z.zero_norm_forward, *forward_args(z, rstd=at(6) + 2))
    refused(z, 2, z.zero_norm_backward, *backward_args(z, gain=at(4) + 1))
    refused(z, 2, z.zero_norm_backward, *backward_args(z, dg=at(7) + 1))
    refused(z, 2, z.zero_norm_backward, *backward_args(z, rstd=at(3) + 2))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, rstd=None))
    refused(z, 2, z.zero_act_weight_grad, *wgrad_args(z, gain=at(3) + 1))
    refused(z, 5, z.zero_norm_forward, mat(z, at(1), 1, 32769), None, None, 1e-5, None,
            mat(z, at(2), 1, 32769), None, None)


def test_null_descriptors(z):
    L = z.lib()
    m, i, c = mat(z, at(1), 10, 64), z.Ids(at(2), 10, 8), ckpt(z, at(3), 10, 64)
    M, I, K = C.byref(m), C.byref(i), C.byref(c)
    assert L.zero_embed_lookup(None, I, 1.0, M, None, None) == 1
    assert L.zero_embed_lookup(M, None, 1.0, M, None, None) == 1
    assert L.zero_embed_lookup(M, I, 1.0, None, None, None) == 1
    assert L.zero_embed_grad(None, I, 1.0, 0, M, None, 0, None, None) == 1
    assert L.zero_embed_grad(M, None, 1.0, 0, M, None, 0, None, None) == 1
    assert L.zero_embed_grad(M, I, 1.0, 0, None, None, 0, None, None) == 1
    assert L.zero_norm_forward(None, None, None, 1e-5, M, M, None, K, None) == 1
    assert L.zero_norm_backward(None, K, at(5), None, None, M, None, 0, None, 0, None) == 1
    assert L.zero_norm_backward(M, None, at(5), None, None, M, None, 0, None, 0, None) == 1
    assert L.zero_norm_backward(M, K, at(5), None, None, None, None, 0, None, 0, None) == 1
    assert L.zero_act_pack(None, K, None) == 1 and L.zero_act_pack(M, None, None) == 1
    assert L.zero_act_unpack(None, M, None) == 1 and L.zero_act_unpack(K, None, None) == 1
    assert L.zero_act_weight_grad(None, K, None, 0, M, None, 0, None) == 1
    assert L.zero_act_weight_grad(M, None, None, 0, M, None, 0, None) == 1
    assert L.zero_act_weight_grad(M, K, None, 0, None, None, 0, None) == 1


def test_overlaps(z):
    inside = at(1) + 64
    refused(z, 1, z.zero_embed_lookup, *lookup_args(z, out=mat(z, inside, 10, 64)))
    refused(z, 1, z.zero_embed_lookup, *lookup_args(z, bad=at(3)))
    refused(z, 1, z.zero_embed_grad, *egrad_args(z, ws=inside))
    refused(z, 1, z.zero_embed_grad, *egrad_args(z, d_out=mat(z, inside, 10, 64)))
    for name in ("h", "y"):
        refused(z, 1, z.zero_norm_forward, *forward_args(z, **{name: mat(z, inside, 10, 64)}))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, y=mat(z, at(1), 10, 64)))   # h may, y may not
    refused(z, 1, z.zero_norm_forward, *forward_args(z, y=mat(z, at(4), 10, 64)))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, c=ckpt(z, at(5), 10, 64)))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, rstd=at(4)))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, dx=mat(z, inside, 10, 64)))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, dx=mat(z, at(2), 10, 64)))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, dg=at(6)))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, ws=at(1)))
    refused(z, 1, z.zero_act_pack, mat(z, at(1), 10, 64), ckpt(z, inside, 10, 64))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=mat(z, inside, 40, 64)))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=mat(z, at(2), 40, 64)))
    # column slices of one buffer that share columns 56..63
    refused(z, 1, z.zero_norm_forward, mat(z, at(1), 10, 64, 128), None, None, 1e-5, None,
            mat(z, at(1) + 112, 10, 64, 128), None, None)


def test_workspaces(z):
    need = z.zero_embed_grad_workspace(10, 100, 64)
    assert need > 0
    refused(z, 1, z.zero_embed_grad, *egrad_args(z, n=need - 1))
    refused(z, 1, z.zero_embed_grad, *egrad_args(z, ws=None))
    refused(z, 2, z.zero_embed_grad, *egrad_args(z, ws=at(5) + 8))
    need = z.zero_norm_backward_workspace(10, 64)
    assert need > 0
    refused(z, 1, z.zero_norm_backward, *backward_args(z, n=need - 1))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, ws=None))
    refused(z, 2, z.zero_norm_backward, *backward_args(z, ws=at(8) + 8))
    need = z.zero_act_weight_grad_workspace(10, 40, 64)
    if need:
        refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, n=need - 1))
        refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, ws=None))
        refused(z, 2, z.zero_act_weight_grad, *wgrad_args(z, ws=at(5) + 8))
    top = 2 ** 64 - 1
    assert z.zero_embed_grad_workspace(1 << 31, 10, 10) == top
    assert z.zero_embed_grad_workspace(10, 1 << 31, 10) == top
    assert z.zero_embed_grad_workspace(10, 10, 1 << 40) == top
    assert z.zero_norm_backward_workspace(10, 32769) == top
    assert z.zero_norm_backward_workspace(0, 64) == 0
    for rows in (1, 100, 10 ** 6, 1 << 40):   # grows to a limit
        assert z.zero_norm_backward_workspace(rows, 64) <= 1216 * 64 * 4


def test_tensors_that_no_descriptor_fits(z):
    for t in (torch.zeros(4, 4), torch.zeros(4, dtype=torch.float16),
              torch.zeros(4, 8, dtype=torch.bfloat16).t(), torch.zeros(4, 4, dtype=torch.int16)):
        with pytest.raises(ValueError):
            z.mat(t)
    for t in (torch.zeros(4), torch.zeros(4, dtype=torch.int16), torch.zeros(8, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            z.ids(t)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    for a, b in ((q, s[:, :1]), (q[:2], s), (q.t(), s), (q.float(), s), (q, s.int())):
        with pytest.raises(ValueError):
            z.act8(a, b)
    m = z.mat(torch.zeros(6, 40, dtype=torch.bfloat16)[:, :33])
    assert (m.rows, m.cols, m.pitch, m.dtype) == (6, 33, 40, z.ZERO_BF16)
    c = z.act8(q[:, :50], s)
    assert (c.rows, c.cols, c.q_pitch, c.scale_pitch) == (4, 50, 64, 2)
    q, s = z.act8_empty(3, 77, device="cpu")
    assert q.shape == (3, 77) and q.stride(0) == 80 and s.shape == (3, 3)


def test_definition_of_the_checkpoint():
    """The tests' own definition: known blocks by hand."""
    x = torch.tensor([[127.0, 1.0, -63.5, 0.5] + [0.0] * 28 + [128.0, -2.0]])
    q, s = ref.pack(x, "bf16")
    assert s.tolist() == [[127, 128]]
    assert q[0, :4].tolist() == [127, 1, -64, 0] and q[0, 32:].tolist() == [64, -1]
    q, s = ref.pack(torch.full((1, 1), 65504.0), "f16")
    assert (int(s), int(q)) == (136, 127)
    q, s = ref.pack(torch.tensor([[float("nan"), 1.0]]), "f16")
    assert int(s) == 255 and not q.any()


def test_header_compiles_as_c(tmp_path):
    """Plain C99 against zero_train.h: the descriptors and a host-only entry point."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "use.c"
    src.write_text("""
#include <stdio.h>
#include "zero_train.h"
int main(void)
{
    zero_mat_t m = {0, 0, 8, 8, ZERO_BF16};
    zero_act8_t c = {0, 0, 0, 8, 16, 1};
    zero_ids_t i = {0, 0, 8};
    printf("%d %d %d %llu %u\\n", (int)zero_act_pack(&m, &c, 0), (int)zero_act_unpack(&c, &m, 0),
           (int)zero_embed_lookup(&m, &i, 1.0f, &m, 0, 0),
           (unsigned long long)zero_norm_backward_workspace(10, 64), ZERO_ACT8_BLOCK);
    return 0;
}
""")
    from zero_sharded_optimizer_02_gb300 import _abi, build
    build.build()
    exe = tmp_path / "use"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                           os.path.join(root, "include"), str(src), _abi.LIB_PATH, "-o", str(exe),
                           "-Wl,-rpath," + os.path.dirname(_abi.LIB_PATH)])
    out = subprocess.check_output([str(exe)], text=True).split()
    assert out[:3] == ["0", "0", "0"] and int(out[3]) > 0 and out[4] == "32"


def test_token_numbers_are_signed_whole_numbers(z):
    """Other elements of 4 or 8 bytes are no token numbers."""
    for dtype in (torch.complex64, torch.uint32, torch.uint64, torch.float32, torch.float64):
        with pytest.raises(ValueError):
            z.ids(torch.zeros(4, dtype=dtype))
    for dtype, size in ((torch.int32, 4), (torch.int64, 8)):
        i = z.ids(torch.zeros(2, 3, dtype=dtype))
        assert (i.count, i.bytes) == (6, size)


def test_vectors_of_another_type_or_size(z):
    """A tensor that is not what the kernels read or write at its address is refused before
    the library sees it: the matrices are at made-up addresses, and nothing is launched."""
    good = dict(gain=torch.zeros(64, dtype=torch.float16), rstd=torch.zeros(10), ws=torch.zeros(1 << 20, dtype=torch.uint8),
                bad=torch.zeros(1, dtype=torch.int32))
    half, wide = torch.zeros(64, dtype=torch.float16), torch.zeros(128, dtype=torch.float16)
    bad_gains = (half.float(), half.bfloat16(), half[:63], wide[::2], half.short())
    bad_rstds = (torch.zeros(10, dtype=torch.float16), torch.zeros(10, dtype=torch.float64), torch.zeros(9),
                 torch.zeros(20)[::2])
    bad_spaces = (good["ws"][:99], torch.zeros(49, dtype=torch.int16), good["ws"][::2])

    def value_error(fn, args):
        with pytest.raises(ValueError):
            fn(*args)

    for g in bad_gains:
        value_error(z.zero_norm_forward, forward_args(z, gain=g))
        value_error(z.zero_norm_backward, backward_args(z, gain=g))
        value_error(z.zero_norm_backward, backward_args(z, dg=g))
        value_error(z.zero_act_weight_grad, wgrad_args(z, gain=g))
    for r in bad_rstds:
        value_error(z.zero_norm_forward, forward_args(z, rstd=r))
        value_error(z.zero_norm_backward, backward_args(z, rstd=r))
    for w in bad_spaces:
        for fn, args in ((z.zero_embed_grad, egrad_args), (z.zero_norm_backward, backward_args),
                         (z.zero_act_weight_grad, wgrad_args)):
            value_error(fn, args(z, ws=w, n=100 if w.is_contiguous() else 1 << 19))
    for b in (torch.zeros(1, dtype=torch.bool), torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.float16)):
        value_error(z.zero_embed_lookup, lookup_args(z, bad=b))
        value_error(z.zero_embed_grad, egrad_args(z, bad=b))
    # what fits reaches the library, which refuses a misaligned matrix here
    off = mat(z, A + 2, 10, 64)
    refused(z, 2, z.zero_norm_forward, *forward_args(z, y=off, gain=good["gain"].view(1, 64), rstd=good["rstd"]))
    refused(z, 2, z.zero_norm_backward, *backward_args(z, dx=off, gain=torch.zeros(70, dtype=torch.float16),
                                                       rstd=good["rstd"].view(1, 10), dg=good["gain"], ws=good["ws"],
                                                       n=1 << 20))
    refused(z, 2, z.zero_embed_lookup, *lookup_args(z, out=off, bad=good["bad"]))
    refused(z, 2, z.zero_embed_grad, *egrad_args(z, d_out=off, bad=good["bad"].long(), ws=good["ws"], n=1 << 20))
    refused(z, 2, z.zero_act_weight_grad, *wgrad_args(z, dy=mat(z, A + 2, 10, 40), gain=good["gain"], ws=good["ws"],
                                                      n=1 << 20))
    # neither is anything asked of an address, or of an object that only has one
    class Address:
        def data_ptr(self):
            return at(3)

    refused(z, 2, z.zero_norm_forward, *forward_args(z, y=off, gain=Address(), rstd=at(6)))
    refused(z, 1, z.zero_norm_forward, *forward_args(z, x=None, gain=good["gain"]))
    refused(z, 1, z.zero_norm_backward, *backward_args(z, dy=None, gain=good["gain"]))
    refused(z, 1, z.zero_act_weight_grad, *wgrad_args(z, dw=None, gain=good["gain"]))
