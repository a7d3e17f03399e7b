"""A small language model trained with the library's operators and its ZeRO step.

    python examples/checkpointed_lm.py [--steps 60] [--dim 256] [--layers 2]

Two emulated data-parallel ranks share one flat 16-bit parameter buffer (the
gathered buffer of ``DataParallelStep``).  For its micro-batch each rank runs

    embedding lookup -> residual blocks -> norm -> tied output layer

and writes its gradient, matrix after matrix, straight into its contribution
row, which the optimizer step then reduces.  (A row holds one shard every
row_pitch elements.  It is the flat gradient if row_pitch is the shard's own
length, so the flat buffer is padded to that.)  Nothing of a block is kept for the backward
pass but 8-bit checkpoints:

  - of the normalised rows (written by the norm itself): they serve the norm's
    backward pass and the weight gradient of the layer behind it;
  - of the hidden layer before its nonlinearity (x sigmoid(x), which is smooth:
    a rectifier's mask would be lost where the checkpoint rounds to zero): the
    activations and the derivative are computed again from it.

The table's gradient is the output layer's weight gradient, onto which the
lookup's gradient is added.  Matrix products with the weights themselves are
torch's, on its current stream, which every operator is therefore given: the
library's own default is the legacy stream, and does not follow torch's.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_sharded_optimizer_02_gb300 as z
from zero_sharded_optimizer_02_gb300.step import DataParallelStep

EPS = 1e-5


class Shapes:
    """The model's matrices and where each lies in the flat buffer (offsets are
    multiples of 8 elements, so every matrix has 16-byte rows), whose length is a
    multiple of 8 for each of nd shards."""

    def __init__(self, vocab: int, dim: int, hidden: int, layers: int, nd: int = 1):
        if dim % 8 or hidden % 8:
            raise ValueError("dim and hidden must be multiples of 8")
        self.vocab, self.dim, self.hidden, self.layers = vocab, dim, hidden, layers
        self.at, n = {}, 0
        named = [("table", vocab, dim)]
        for k in range(layers):
            named += [(f"gain{k}", 1, dim), (f"up{k}", hidden, dim), (f"down{k}", dim, hidden)]
        for name, rows, cols in named + [("gain_out", 1, dim)]:
            self.at[name] = (n, rows, cols)
            n += -(-rows * cols // 8) * 8
        self.psi = -(-n // (8 * nd)) * 8 * nd

    def view(self, flat: torch.Tensor, name: str) -> torch.Tensor:
        n, rows, cols = self.at[name]
        return flat[n:n + rows * cols].view(rows, cols)


class Workspaces:
    """One workspace for every operator of a micro-batch, run one after another."""

    def __init__(self, s: Shapes, tokens: int):
        n = max(z.zero_norm_backward_workspace(tokens, s.dim),
                z.zero_embed_grad_workspace(tokens, s.vocab, s.dim),
                z.zero_act_weight_grad_workspace(tokens, s.hidden, s.dim),
                z.zero_act_weight_grad_workspace(tokens, s.dim, s.hidden),
                z.zero_act_weight_grad_workspace(tokens, s.vocab, s.dim))
        self.buf = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    @property
    def args(self):
        return self.buf, self.buf.numel()


def loss_and_grads(s: Shapes, params: torch.Tensor, row: torch.Tensor, tokens: torch.Tensor,
                   targets: torch.Tensor, ws: Workspaces) -> torch.Tensor:
    """The mean cross-entropy of one micro-batch; its gradient is stored in `row`."""
    t, d = tokens.numel(), s.dim
    st = torch.cuda.current_stream()      # torch's own work between the operators goes there
    scale = math.sqrt(d)
    # activations: rows on 16-byte boundaries, whatever their width
    like = lambda cols: torch.empty(t, -(-cols // 8) * 8, dtype=params.dtype,     # noqa: E731
                                    device="cuda")[:, :cols]
    p = lambda name: s.view(params, name)                                         # noqa: E731
    g = lambda name: z.mat(s.view(row, name))                                     # noqa: E731
    ids = z.ids(tokens)

    # forward: x is what the last block added, h the residual stream so far
    kept = []
    x, h = like(d), None
    z.zero_embed_lookup(z.mat(p("table")), ids, scale, z.mat(x), stream=st)
    for k in range(s.layers + 1):
        gain = p("gain_out" if k == s.layers else f"gain{k}")
        y, rstd = like(d), torch.empty(t, device="cuda")
        normed = z.act8_empty(t, d)
        new_h = h if h is not None else like(d)          # the sum takes the stream's place
        z.zero_norm_forward(z.mat(x), z.mat(h) if h is not None else None, gain, EPS,
                            z.mat(new_h), z.mat(y), rstd, z.act8(*normed), st)
        h = new_h
        if k == s.layers:
            break
        u = y @ p(f"up{k}").t()
        hidden = z.act8_empty(t, s.hidden)
        z.zero_act_pack(z.mat(u), z.act8(*hidden), st)
        x = torch.nn.functional.silu(u) @ p(f"down{k}").t()
        kept.append((normed, rstd, hidden))              # y, u and h are not kept
        del y, u
    logits = (y @ p("table").t()).float()
    loss = torch.nn.functional.cross_entropy(logits, targets)

    # backward: the output layer, whose weight is the table
    soft = torch.softmax(logits, 1)
    soft[torch.arange(t, device="cuda"), targets] -= 1
    d_logits = like(s.vocab)
    d_logits.copy_(soft / t)
    z.zero_act_weight_grad(z.mat(d_logits), z.act8(*normed), p("gain_out"), False, g("table"), *ws.args, stream=st)
    d_y, d_h = d_logits @ p("table"), like(d)
    z.zero_norm_backward(z.mat(d_y), z.act8(*normed), rstd, p("gain_out"), None, z.mat(d_h),
                         s.view(row, "gain_out"), False, *ws.args, stream=st)
    for k in reversed(range(s.layers)):                  # d_h: of h behind the block, and of x
        normed, rstd, hidden = kept[k]
        u = like(s.hidden)
        z.zero_act_unpack(z.act8(*hidden), z.mat(u), st)
        open_ = torch.sigmoid(u.float())
        a = (u * open_).to(u.dtype)
        z.zero_act_pack(z.mat(a), z.act8(*hidden), st)   # in the place of u's
        z.zero_act_weight_grad(z.mat(d_h), z.act8(*hidden), None, False, g(f"down{k}"), *ws.args, stream=st)
        d_u = ((d_h @ p(f"down{k}")) * (open_ + a * (1 - open_))).to(u.dtype)
        z.zero_act_weight_grad(z.mat(d_u), z.act8(*normed), p(f"gain{k}"), False, g(f"up{k}"), *ws.args, stream=st)
        d_y = d_u @ p(f"up{k}")
        z.zero_norm_backward(z.mat(d_y), z.act8(*normed), rstd, p(f"gain{k}"), z.mat(d_h), z.mat(d_h),
                             s.view(row, f"gain{k}"), False, *ws.args, stream=st)
    z.zero_embed_grad(z.mat(d_h), ids, scale, True, g("table"), *ws.args, stream=st)
    return loss


def make_group(s: Shapes, nd: int, lr: float, seed: int = 0) -> DataParallelStep:
    """The ranks' sharded fp32 state, and the 16-bit parameters gathered from it."""
    dps = DataParallelStep(s.psi, nd, range(nd), "bf16",
                           dict(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01), 1.0,
                           1 << 20)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    flat = torch.zeros(s.psi, device="cuda")
    for name, (_, rows, cols) in s.at.items():
        view = s.view(flat, name)
        if name.startswith("gain"):
            view.fill_(1.0)
        else:
            view.normal_(0.0, 1.0 / math.sqrt(cols), generator=gen)
    st = torch.cuda.current_stream()
    for r in dps.ranks:
        n, b = int(dps.layouts[r].length), int(dps.layouts[r].begin)
        zero = torch.zeros(n, device="cuda")
        dps.state[r].load(flat[b:b + n], zero, zero)
        master = dps.state[r].tensors()[0]
        z.zero_gather_params_shard(master, n, dps.gathered_view(), b, "bf16", st)
    return dps


def train(steps: int = 60, vocab: int = 1000, dim: int = 256, hidden: int = 512, layers: int = 2,
          tokens: int = 512, nd: int = 2, lr: float = 2e-3, say=print) -> list:
    """Trains on sequences whose next token is a fixed permutation of the last;
    returns the mean loss of every step."""
    s = Shapes(vocab, dim, hidden, layers, nd)
    dps = make_group(s, nd, lr)
    pitch = int(dps.layouts[0].row_pitch)
    assert nd * pitch == s.psi            # the shards of a row lie end to end
    rows = torch.zeros(nd, s.psi, dtype=torch.bfloat16, device="cuda")
    desc = {r: z.grads(rows, nd * pitch, r * pitch, nd, "bf16") for r in dps.ranks}
    ws = Workspaces(s, tokens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    losses = []
    for step in range(steps):
        total = 0.0
        for j in range(nd):
            toks = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
            total = total + loss_and_grads(s, dps.gathered_view()[:s.psi], rows[j], toks, follow[toks], ws)
        if dps.step(desc):
            say(f"step {step}: a nonfinite gradient, skipped on every rank")
        losses.append(float(total) / nd)
        if step % 10 == 0 or step + 1 == steps:
            say(f"step {step:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    train(steps=a.steps, dim=a.dim, hidden=2 * a.dim, layers=a.layers)
