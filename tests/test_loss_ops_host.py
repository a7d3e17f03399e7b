"""Refusals of the losses behind the output layer, without a GPU: every invalid
argument is reported on the host and nothing is launched.  The addresses are
never dereferenced: each call fails validation before any CUDA call, or has
nothing to do."""
import pytest
import torch

A = 1 << 20          # a 16-byte aligned address
STEP = 1 << 30       # further apart than any buffer below
T, V, K = 10, 64, 5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def z():
    from zero_sharded_optimizer_02_gb300 import build
    build.build()
    import zero_sharded_optimizer_02_gb300 as z
    return z


def at(k):
    return A + k * STEP


def mat(z, where, rows=T, cols=V, pitch=None, dtype=None):
    return z.Mat(where, rows, cols, -(-cols // 8) * 8 if pitch is None else pitch, z.ZERO_F16 if dtype is None else dtype)


def refused(z, status, fn, args):
    with pytest.raises(z.ZeroError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def args_of(z, name, **kw):
    ids = lambda k: z.Ids(at(k), T, 8)   # noqa: E731
    a = dict(
        logprob=dict(logits=mat(z, at(1)), targets=ids(2), temp=1.0, logp=at(3), lse=at(4), bad=at(5)),
        backward=dict(logits=mat(z, at(1)), targets=ids(2), temp=1.0, d_logp=at(3), d=mat(z, at(4)), bad=at(5)),
        distill=dict(logits=mat(z, at(1)), top=mat(z, at(6), cols=K), top_ids=z.Ids(at(7), T * K, 4), temp=1.0, soft=0.5,
                     targets=ids(2), hard=0.5, weight=at(8), scale=1.0, loss=at(9), d=mat(z, at(4)), bad=at(5)),
        policy=dict(logits=mat(z, at(1)), targets=ids(2), temp=1.0, old=at(6), ref=at(7), adv=at(8), weight=at(9), low=0.2,
                    high=0.2, kl=0.1, scale=1.0, loss=at(10), logp=at(11), d=mat(z, at(4)), bad=at(5)),
        pref=dict(logits=mat(z, at(1)), targets=ids(2), starts=z.Ids(at(6), 5, 8), ref=at(7), beta=0.1, smoothing=0.0, scale=1.0,
                  loss=at(8), reward=at(9), logp=at(10), d=mat(z, at(4)), ws=at(11), n=1 << 20, bad=at(5)))[name]
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


FNS = dict(logprob="zero_token_logprob", backward="zero_token_logprob_backward", distill="zero_distill_loss",
           policy="zero_policy_loss", pref="zero_preference_loss")
WITH_GRAD = ("backward", "distill", "policy", "pref")


def bad(z, name, status, **kw):
    refused(z, status, getattr(z, FNS[name]), args_of(z, name, **kw))


@pytest.mark.parametrize("name", FNS)
def test_logits(z, name):
    for m, status in ((mat(z, A + 2), 2), (mat(z, at(1), pitch=65), 2), (mat(z, at(1), pitch=56), 1), (mat(z, at(1), dtype=2), 1),
                      (mat(z, None), 1), (mat(z, at(1), pitch=1 << 57), 1), (mat(z, at(1), rows=9), 1),
                      (mat(z, at(1), cols=0, pitch=0), 1)):
        bad(z, name, status, logits=m)
    bad(z, name, 1, logits=None)
    wide = z.ZERO_LOSS_MAX_VOCAB + 1
    kw = {"d": mat(z, at(4), cols=wide)} if name in WITH_GRAD else {}
    bad(z, name, 5, logits=mat(z, at(1), cols=wide), **kw)


@pytest.mark.parametrize("name", WITH_GRAD)
def test_gradients(z, name):
    for m, status in ((mat(z, A + 2), 2), (mat(z, at(4), pitch=65), 2), (mat(z, at(4), rows=9), 1), (mat(z, at(4), cols=63), 1),
                      (mat(z, at(4), dtype=z.ZERO_BF16), 1), (mat(z, None), 1)):
        bad(z, name, status, d=m)
    # in the logits' place with another pitch, or a part of them
    bad(z, name, 1, d=mat(z, at(1), pitch=72))
    bad(z, name, 1, d=mat(z, at(1) + 16))
    bad(z, name, 1, logits=mat(z, at(1), pitch=72), d=mat(z, at(1) + 16, pitch=72))


@pytest.mark.parametrize("name", FNS)
def test_targets(z, name):
    for i, status in ((z.Ids(at(2), 9, 8), 1), (z.Ids(at(2), T, 2), 1), (z.Ids(at(2) + 4, T, 8), 2), (z.Ids(None, T, 8), 1),
                      (z.Ids(at(2), 1 << 31, 8), 5)):
        bad(z, name, status, targets=i)
    bad(z, name, 1, targets=None)          # distill: its hard part is wanted


@pytest.mark.parametrize("name", ["logprob", "backward", "distill", "policy"])
def test_temperatures(z, name):
    for t in (0.0, -1.0, NAN, INF, 2.0 ** -21, 2.0 ** 21):
        bad(z, name, 1, temp=t)


@pytest.mark.parametrize("name", ["distill", "policy", "pref"])
def test_scales(z, name):
    for s in (NAN, INF, -INF):
        bad(z, name, 1, scale=s)


def test_other_numbers(z):
    for x in (NAN, INF):
        bad(z, "distill", 1, soft=x)
        bad(z, "distill", 1, hard=x)
        bad(z, "policy", 1, kl=x)
        bad(z, "policy", 1, low=x)
        bad(z, "policy", 1, high=x)
        bad(z, "pref", 1, beta=x)
        bad(z, "pref", 1, smoothing=x)
    bad(z, "policy", 1, low=-0.1)
    bad(z, "policy", 1, low=1.1)
    bad(z, "policy", 1, high=-0.1)
    bad(z, "pref", 1, smoothing=-0.1)
    bad(z, "pref", 1, smoothing=1.1)


def test_nothing_wanted(z):
    bad(z, "logprob", 1, logp=None, lse=None)
    bad(z, "backward", 1, d=None)
    bad(z, "distill", 1, loss=None, d=None)
    bad(z, "policy", 1, loss=None, logp=None, d=None)
    bad(z, "pref", 1, loss=None)


def test_missing_vectors(z):
    bad(z, "backward", 1, d_logp=None)
    bad(z, "policy", 1, old=None)
    bad(z, "policy", 1, adv=None)
    bad(z, "policy", 1, ref=None)          # its KL term is wanted


def test_alignment_of_vectors(z):
    for name, keys in (("logprob", ["logp", "lse", "bad"]), ("backward", ["d_logp", "bad"]), ("distill", ["weight", "loss", "bad"]),
                       ("policy", ["old", "ref", "adv", "weight", "loss", "logp", "bad"]),
                       ("pref", ["ref", "loss", "reward", "logp", "bad"])):
        for k in keys:
            bad(z, name, 2, **{k: at(20) + 2})
    bad(z, "pref", 2, ws=at(20) + 8)


def test_teachers(z):
    bad(z, "distill", 1, top=None)
    bad(z, "distill", 1, top_ids=None)
    for m, status in ((mat(z, A + 2, cols=K), 2), (mat(z, at(6), rows=9, cols=K), 1), (mat(z, at(6), cols=K, dtype=z.ZERO_BF16), 1),
                      (mat(z, at(6), cols=K, pitch=9), 2), (mat(z, None, cols=K), 1), (mat(z, at(6), cols=K + 1), 1)):
        bad(z, "distill", status, top=m)
    wide = z.ZERO_DISTILL_MAX_TOP + 1
    bad(z, "distill", 5, top=mat(z, at(6), cols=wide), top_ids=z.Ids(at(7), T * wide, 4))
    for i, status in ((z.Ids(at(7), T * K - 1, 4), 1), (z.Ids(at(7) + 2, T * K, 4), 2), (z.Ids(at(7), T * K, 3), 1),
                      (z.Ids(None, T * K, 4), 1)):
        bad(z, "distill", status, top_ids=i)


def test_starts_and_workspace(z):
    for i, status in ((z.Ids(at(6), 4, 8), 1), (z.Ids(at(6), 0, 8), 1), (z.Ids(at(6) + 4, 5, 8), 2), (z.Ids(None, 5, 8), 1),
                      (z.Ids(at(6), 5, 1), 1), (None, 1)):
        bad(z, "pref", status, starts=i)
    need = z.zero_preference_loss_workspace(T, 2)
    assert need >= 8 * T
    bad(z, "pref", 1, n=need - 1)
    bad(z, "pref", 1, ws=None)
    assert z.zero_preference_loss_workspace(1 << 32, 1) == 2 ** 64 - 1


def test_overlaps(z):
    x, d = at(1), at(4)
    for name, outs in (("logprob", ["logp", "lse", "bad"]), ("backward", ["bad"]), ("distill", ["loss", "bad"]),
                       ("policy", ["loss", "logp", "bad"]), ("pref", ["loss", "reward", "logp", "ws", "bad"])):
        for k in outs:
            bad(z, name, 1, **{k: x + 128})                  # an output inside the logits
            bad(z, name, 1, **{k: at(2) + (0 if k == "ws" else 8)})   # and inside the targets
            if name in WITH_GRAD:
                bad(z, name, 1, **{k: d + 128})              # and inside the gradient
    bad(z, "backward", 1, d_logp=d + 64)
    bad(z, "policy", 1, old=at(11))
    bad(z, "policy", 1, ref=at(10) + 4)
    bad(z, "distill", 1, top=mat(z, d, cols=K))
    bad(z, "distill", 1, weight=at(9))
    bad(z, "pref", 1, ref=at(11) + 16)
    bad(z, "pref", 1, reward=at(8) + 4)


def test_calls_without_rows(z):
    """Nothing to do: no CUDA call, whatever the addresses."""
    none = z.Ids(None, 0, 8)
    m = mat(z, at(1), rows=0)
    z.zero_token_logprob(m, none, 1.0, at(3))
    z.zero_token_logprob_backward(m, none, 1.0, at(3), mat(z, at(4), rows=0))
    z.zero_distill_loss(m, None, None, 1.0, 0.0, none, 1.0, None, 1.0, at(3), None)
    z.zero_policy_loss(m, none, 1.0, None, None, None, None, 0.2, 0.2, 0.0, 1.0, at(3))
    z.zero_preference_loss(m, none, z.Ids(at(6), 1, 8), None, 0.1, 0.0, 1.0, None, None, None, None, at(7), 1 << 20)


def test_vectors_of_another_type_or_size(z):
    """A tensor that is not what the kernels read or write at its address is refused before the library sees it."""
    f = torch.zeros(T)
    for v in (f.half(), f.double(), f[:T - 1], torch.zeros(2 * T)[::2], f.int()):
        for name, keys in (("logprob", ["logp", "lse"]), ("backward", ["d_logp"]), ("distill", ["weight", "loss"]),
                           ("policy", ["old", "ref", "adv", "weight", "loss", "logp"]), ("pref", ["ref", "logp"])):
            for k in keys:
                with pytest.raises(ValueError):
                    getattr(z, FNS[name])(*args_of(z, name, **{k: v}))
    for k, n in (("loss", 2), ("reward", 4)):
        with pytest.raises(ValueError):
            z.zero_preference_loss(*args_of(z, "pref", **{k: torch.zeros(n - 1)}))
    with pytest.raises(ValueError):
        z.zero_preference_loss(*args_of(z, "pref", ws=torch.zeros(99, dtype=torch.uint8), n=100))
    for name in FNS:
        with pytest.raises(ValueError):
            getattr(z, FNS[name])(*args_of(z, name, bad=torch.zeros(1, dtype=torch.int16)))


def test_header_compiles_as_c(tmp_path):
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
    zero_ids_t i = {0, 0, 8};
    float out[1];
    printf("%d %d %d %llu %u %u\\n", (int)zero_token_logprob(&m, &i, 1.0f, out, 0, 0, 0),
           (int)zero_distill_loss(&m, 0, 0, 1.0f, 0.0f, &i, 1.0f, 0, 1.0f, out, 0, 0, 0),
           (int)zero_policy_loss(&m, &i, 0.0f, 0, 0, 0, 0, 0.2f, 0.2f, 0.0f, 1.0f, out, 0, 0, 0, 0),
           (unsigned long long)zero_preference_loss_workspace(10, 2), ZERO_LOSS_MAX_VOCAB, ZERO_DISTILL_MAX_TOP);
    return 0;
}
""")
    from zero_sharded_optimizer_02_gb300 import _abi, build
    build.build()
    exe = tmp_path / "use"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(root, "include"),
                           str(src), _abi.LIB_PATH, "-o", str(exe), "-Wl,-rpath," + os.path.dirname(_abi.LIB_PATH)])
    out = subprocess.check_output([str(exe)], text=True).split()
    assert out[:3] == ["0", "0", "1"] and int(out[3]) > 0 and out[4:] == ["393216", "256"]
