"""Workloads of the losses behind the output layer of a language model.

The output layer of a training step gives one row of 16-bit logits a token, as
wide as the vocabulary.  The operators here turn those rows into a loss and
into the gradient that goes back through the layer:

  logp       log-probability of each token's target (scoring with a frozen model)
  logp_grad  the gradient of those, from the gradient of every log-probability
  distill    distillation from a teacher's top logits, mixed with the ordinary
             cross-entropy of the target (which alone is the ordinary loss)
  policy     a clipped policy loss with a KL term to a reference model
  pref       a preference loss on pairs of sequences (paired log ratios)

With p = softmax(z / T) of a row z, target y and lp = log p[y]:

  distill    q = softmax(teacher / T) over the top entries that are present;
             loss = soft * T^2 * sum q (log q - log p) - hard * log softmax(z)[y]
  policy     r = exp(lp - old), d = ref - lp;
             loss = weight * (-min(r A, clip(r, 1 - lo, 1 + hi) A) + kl (exp(d) - d - 1))
  pref       s of a sequence = sum of lp - ref over its tokens, m = beta (s_chosen - s_rejected);
             loss = -(1 - eps) log sigmoid(m) - eps log sigmoid(-m)

A row whose target is negative is padding: its loss, log-probability and
gradient are zero and its logits are not looked at.  Gradients are those of
the sum of the losses times `scale`.

Every case names its operator in ``"op"``; ``run`` does one pass of it, either
in plain torch operations in 32 bits or through the framework's entry points
(``own``).
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_ELEMS = 600_000_000   # most logits of a drawn case (the largest listed one has 823,410,688)


def listed():
    return [
        # One token scored in a loop: what it costs is latency.
        dict(name="logp_token", op="logp", tokens=1, vocab=50257, live=50257, dtype="bf16", temp=1.0, pad=0.0),
        # A long micro-batch scored with the frozen model, a quarter of it prompt.
        dict(name="logp_batch", op="logp", tokens=16384, vocab=50257, live=50257, dtype="f16", temp=0.7, pad=0.25),
        # The gradient for a loss of the user's own on the log-probabilities; odd sizes.
        dict(name="logp_grad_odd", op="logp_grad", tokens=1021, vocab=32001, live=32001, dtype="bf16", temp=1.0, pad=0.1),
        # A few tokens of an online student.
        dict(name="distill_few", op="distill", tokens=7, vocab=50257, live=50257, dtype="bf16", top=8, ids=32, temp=1.0, soft=1.0,
             hard=0.0, pad=0.0),
        # A short, ragged batch: an odd number of teacher entries, some of them absent, padding.
        dict(name="distill_odd", op="distill", tokens=333, vocab=50257, live=50257, dtype="f16", top=17, ids=64, temp=2.0, soft=0.5,
             hard=0.5, pad=0.06),
        # A training micro-batch whose vocabulary is padded to 64s: softmax at two temperatures.
        dict(name="distill_batch", op="distill", tokens=8192, vocab=50304, live=50257, dtype="f16", top=64, ids=32, temp=2.0,
             soft=0.9, hard=0.1, pad=0.0),
        # The ordinary loss of a long micro-batch: cross-entropy and its gradient.
        dict(name="xent_batch", op="distill", tokens=16384, vocab=50257, live=50257, dtype="bf16", top=0, ids=64, temp=1.0, soft=0.0,
             hard=1.0, pad=0.0),
        # One short completion in a policy step.
        dict(name="policy_few", op="policy", tokens=64, vocab=50257, live=50257, dtype="bf16", temp=1.0, kl=0.05, weight=False,
             pad=0.0),
        # A policy step's micro-batch: prompts and padding are 30 percent of its rows.
        dict(name="policy_batch", op="policy", tokens=16384, vocab=50257, live=50257, dtype="bf16", temp=1.0, kl=0.02, weight=True,
             pad=0.3),
        # A large vocabulary, sampled at a temperature, no KL term.
        dict(name="policy_wide", op="policy", tokens=4096, vocab=131072, live=131072, dtype="f16", temp=0.8, kl=0.0, weight=False,
             pad=0.0),
        # Two short pairs.
        dict(name="pref_few", op="pref", tokens=181, vocab=50257, live=50257, dtype="bf16", pairs=2, eps=0.0, ref=True, pad=0.1),
        # A micro-batch of pairs of some 1,000 tokens a sequence, with prompts left out and label smoothing.
        dict(name="pref_batch", op="pref", tokens=16384, vocab=50257, live=50257, dtype="f16", pairs=8, eps=0.1, ref=True, pad=0.2),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "distill", "distill", "policy", "pref"])
    vocab = _log(rng, 1000, 131072)
    if rng.random() < 0.5:
        vocab = max(64, vocab // 64 * 64)
    tokens = _log(rng, 1, min(16384, _ELEMS // vocab))
    c = dict(op=op, tokens=tokens, vocab=vocab, live=vocab - rng.choice([0, 0, 0, 47, 5]), dtype=rng.choice(["f16", "bf16"]),
             pad=rng.choice([0.0, 0.1, 0.4]))
    if op in ("logp", "logp_grad", "policy"):
        c["temp"] = rng.choice([1.0, 0.7, 1.3])
    if op == "distill":
        c["top"] = rng.choice([0, _log(rng, 1, 256), _log(rng, 1, 256)])
        c["ids"] = rng.choice([32, 64])
        c["temp"] = rng.choice([1.0, 1.0, 2.0, 4.0]) if c["top"] else 1.0
        c["soft"], c["hard"] = rng.choice([(1.0, 0.0), (0.9, 0.1), (0.5, 0.5)]) if c["top"] else (0.0, 1.0)
    if op == "policy":
        c["kl"], c["weight"] = rng.choice([0.0, 0.02, 0.1]), rng.random() < 0.5
    if op == "pref":
        c["pairs"] = min(_log(rng, 1, 64), max(1, tokens // 4))
        c["eps"], c["ref"] = rng.choice([0.0, 0.1]), rng.random() < 0.8
    return c


# -- inputs --------------------------------------------------------------------

_LOW, _HIGH, _BETA = 0.2, 0.28, 0.1


def _matrix(rows, cols, dtype):
    """An activation matrix whose rows start on 16-byte boundaries, as the framework lays its rows out."""
    return torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def _rows_at_once(vocab):
    return max(1, (1 << 27) // vocab)


def _logits(g, c, targets):
    """Rows of logits as a trained model has them: targets of every probability from 1e-6 to almost 1, and the columns that
    only pad the vocabulary at -inf."""
    t, v = c["tokens"], c["vocab"]
    out = _matrix(t, v, _TYPES[c["dtype"]])
    boost = 18.0 * torch.rand(t, generator=g, device="cuda")
    for a in range(0, t, _rows_at_once(v)):
        b = min(t, a + _rows_at_once(v))
        x = 2.0 * torch.randn(b - a, v, generator=g, device="cuda")
        x[torch.arange(b - a, device="cuda"), targets[a:b].clamp(min=0)] += boost[a:b]
        x[:, c["live"]:] = -math.inf
        out[a:b].copy_(x)
    return out


def _model_logp(logits, targets, temp):
    """Log-probabilities of the targets as another run of the model gives them."""
    parts = []
    for a in range(0, logits.shape[0], _rows_at_once(logits.shape[1])):
        x = logits[a:a + _rows_at_once(logits.shape[1])].float() / temp
        y = targets[a:a + x.shape[0]].clamp(min=0)
        parts.append(x.gather(1, y[:, None])[:, 0] - torch.logsumexp(x, 1))
    return torch.cat(parts)


def _teacher(g, c, logits, targets):
    """A teacher's top logits and their numbers, as it sorted them: the student's own largest ones under noise, the target
    often among them; of one row in eight the last entries are absent (-1)."""
    t, k = c["tokens"], c["top"]
    top, ids = _matrix(t, k, logits.dtype), torch.empty(t, k, dtype=torch.int64, device="cuda")
    for a in range(0, t, _rows_at_once(c["vocab"])):
        b = min(t, a + _rows_at_once(c["vocab"]))
        x = logits[a:b].float() + torch.randn(b - a, c["vocab"], generator=g, device="cuda")
        values, ids[a:b] = torch.topk(x, k, dim=1)
        top[a:b].copy_(values)
    short = torch.rand(t, generator=g, device="cuda") < 0.125
    keep = 1 + (torch.rand(t, generator=g, device="cuda") * k).long()
    ids[short[:, None] & (torch.arange(k, device="cuda") >= keep[:, None])] = -1
    return top, ids.to(torch.int32 if c["ids"] == 32 else torch.int64).contiguous()


def _starts(g, c):
    """Where the sequences of the pairs start, ragged; the last entry is the end of the last one, and a few rows of the
    batch may lie behind it."""
    n = 2 * c["pairs"]
    cuts = 0.5 + torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ends = torch.cumsum(cuts, 0) / cuts.sum() * (c["tokens"] - (c["tokens"] > 64) * 5)
    return torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), ends]).round().long()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    op, t = c["op"], c["tokens"]
    rand = lambda: torch.randn(t, generator=g, device="cuda")   # noqa: E731
    s = {"case": c, "scale": (1024.0 if c["dtype"] == "f16" else 1.0) / t}   # f16 gradients are loss-scaled
    s["targets"] = torch.randint(0, c["live"], (t,), generator=g, device="cuda")
    if c["pad"]:
        s["targets"][torch.rand(t, generator=g, device="cuda") < c["pad"]] = -1
    s["logits"] = _logits(g, c, s["targets"])
    if op == "logp_grad":
        s["d_logp"] = rand() * s["scale"]
    if op == "distill" and c["top"]:
        s["top"], s["top_ids"] = _teacher(g, c, s["logits"], s["targets"])
    if op == "policy":
        lp = _model_logp(s["logits"], s["targets"], c["temp"])
        step = 0.15 * rand()          # how far the policy has moved since the sampling; not onto the clip's very borders,
        for border in (math.log(1 - _LOW), math.log(1 + _HIGH)):   # where the slope is not defined
            step = torch.where((step - border).abs() < 1e-3, step + 4e-3, step)
        s["old"], s["ref"] = lp - step, lp + 0.2 * rand()
        s["advantage"] = rand()
        s["weight"] = 0.2 + torch.rand(t, generator=g, device="cuda") if c["weight"] else None
    if op == "pref":
        s["starts"] = _starts(g, c)
        s["ref"] = None
        if c["ref"]:
            s["ref"] = _model_logp(s["logits"], s["targets"], 1.0) + 0.3 * rand()
    if own:
        s["call"] = _handles(s, c)
    return s


def _handles(s, c):
    """What a user's program sets up once for its buffers: the output buffers and workspaces, and the descriptors of the
    buffers that it passes with every step."""
    import zero_sharded_optimizer_02_gb300 as z
    op, t = c["op"], c["tokens"]
    h = {"z": z, "logits": z.mat(s["logits"]), "targets": z.ids(s["targets"])}
    if op != "logp":
        s["d_logits"] = _matrix(t, c["vocab"], s["logits"].dtype)
        h["d_logits"] = z.mat(s["d_logits"])
    if op in ("logp", "policy", "pref"):
        s["logp"] = torch.empty(t, device="cuda")
    if op == "logp":
        s["lse"] = torch.empty(t, device="cuda")
    if op in ("distill", "policy"):
        s["loss"] = torch.empty(t, device="cuda")
    if op == "distill":
        h["top"] = z.mat(s["top"]) if c["top"] else None
        h["top_ids"] = z.ids(s["top_ids"]) if c["top"] else None
    if op == "pref":
        s["loss"] = torch.empty(c["pairs"], device="cuda")
        s["reward"] = torch.empty(2 * c["pairs"], device="cuda")
        h["starts"] = z.ids(s["starts"])
        h["ws"] = torch.empty(max(16, z.zero_preference_loss_workspace(t, c["pairs"])), dtype=torch.uint8, device="cuda")
    return h


# -- one pass ------------------------------------------------------------------


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c, h = s["case"], s["call"]
    z, op = h["z"], c["op"]
    if op == "logp":
        z.zero_token_logprob(h["logits"], h["targets"], c["temp"], s["logp"], s["lse"])
        return {"logp": s["logp"], "lse": s["lse"]}
    if op == "logp_grad":
        z.zero_token_logprob_backward(h["logits"], h["targets"], c["temp"], s["d_logp"], h["d_logits"])
        return {"d_logits": s["d_logits"]}
    if op == "distill":
        z.zero_distill_loss(h["logits"], h["top"], h["top_ids"], c["temp"], c["soft"], h["targets"], c["hard"], None, s["scale"],
                            s["loss"], h["d_logits"])
        return {"loss": s["loss"], "d_logits": s["d_logits"]}
    if op == "policy":
        z.zero_policy_loss(h["logits"], h["targets"], c["temp"], s["old"], s["ref"], s["advantage"], s["weight"], _LOW, _HIGH,
                           c["kl"], s["scale"], s["loss"], s["logp"], h["d_logits"])
        return {"loss": s["loss"], "logp": s["logp"], "d_logits": s["d_logits"]}
    z.zero_preference_loss(h["logits"], h["targets"], h["starts"], s["ref"], _BETA, c["eps"], s["scale"], s["loss"], s["reward"],
                           s["logp"], h["d_logits"], h["ws"], h["ws"].numel())
    return {"loss": s["loss"], "reward": s["reward"], "logp": s["logp"], "d_logits": s["d_logits"]}


def _softmax(x):
    """Probabilities of the rows of x, in place, and the logarithm of the sum of the exponentials."""
    top = x.amax(1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    return x.div_(total), lse


def _plain_logp(s, temp):
    """Rows that are there, their log-probabilities (0 for the others), probabilities and sums."""
    there = s["targets"] >= 0
    y = s["targets"].clamp(min=0)
    x = s["logits"].float() / temp
    at = x.gather(1, y[:, None])[:, 0]
    p, lse = _softmax(x)
    zero = torch.zeros_like(lse)
    return there, y, torch.where(there, at - lse, zero), p, torch.where(there, lse, zero)


def _to_logits(p, y, there, slope, dtype):
    """slope[row] * (one at the target - p), rounded; rows that are not there are zero.  Overwrites p."""
    slope = torch.where(there, slope, torch.zeros_like(slope))[:, None]
    p.mul_(-slope)
    p.scatter_add_(1, y[:, None], slope)
    p.masked_fill_(~there[:, None], 0.0)
    return p.to(dtype)


def _plain_distill(s, c, dtype):
    t = c["tokens"]
    there, y = s["targets"] >= 0, s["targets"].clamp(min=0)
    loss = torch.zeros(t, device="cuda")
    grad = torch.zeros(t, c["vocab"], device="cuda")
    if c["top"]:
        here = s["top_ids"] >= 0
        ids = s["top_ids"].clamp(min=0).long()
        taught = torch.where(here, s["top"].float() / c["temp"], torch.full((), -math.inf, device="cuda"))
        q, q_lse = _softmax(taught.clone())
        x = s["logits"].float() / c["temp"]
        at = x.gather(1, ids)
        p, lse = _softmax(x)
        ratio = (taught - q_lse[:, None]) - (at - lse[:, None])
        loss += c["soft"] * c["temp"] ** 2 * torch.where(q > 0, q * ratio, torch.zeros_like(q)).sum(1)
        grad.add_(p, alpha=c["soft"] * c["temp"])
        grad.scatter_add_(1, ids, q * (-c["soft"] * c["temp"]))
        del p, x
    if c["hard"]:
        x = s["logits"].float()
        at = x.gather(1, y[:, None])[:, 0]
        p, lse = _softmax(x)
        loss += c["hard"] * (lse - at)
        grad.add_(p, alpha=c["hard"])
        grad.scatter_add_(1, y[:, None], torch.full((t, 1), -c["hard"], device="cuda"))
    grad.mul_(s["scale"]).masked_fill_(~there[:, None], 0.0)
    return {"loss": torch.where(there, loss, torch.zeros_like(loss)), "d_logits": grad.to(dtype)}


def _run_plain(s):
    c = s["case"]
    op, dtype = c["op"], _TYPES[c["dtype"]]
    if op == "distill":
        return _plain_distill(s, c, dtype)
    temp = c.get("temp", 1.0)
    there, y, lp, p, lse = _plain_logp(s, temp)
    if op == "logp":
        return {"logp": lp, "lse": lse}
    if op == "logp_grad":
        return {"d_logits": _to_logits(p, y, there, s["d_logp"] / temp, dtype)}
    if op == "policy":
        a = s["advantage"].double()
        r = torch.exp(lp.double() - s["old"])
        d = s["ref"].double() - lp
        kept, cut = r * a, r.clamp(1 - _LOW, 1 + _HIGH) * a
        loss = c["kl"] * (torch.exp(d) - d - 1) - torch.minimum(kept, cut)
        slope = c["kl"] * (1 - torch.exp(d)) - torch.where(kept <= cut, kept, torch.zeros_like(kept))
        if s["weight"] is not None:
            loss, slope = loss * s["weight"], slope * s["weight"]
        loss = torch.where(there, loss, torch.zeros_like(loss)).float()
        return {"loss": loss, "logp": lp, "d_logits": _to_logits(p, y, there, (slope * (s["scale"] / temp)).float(), dtype)}
    # pref: sums over sequences are long
    rows = torch.arange(c["tokens"], device="cuda")
    seq = torch.searchsorted(s["starts"], rows, right=True) - 1
    there = there & (seq < 2 * c["pairs"])
    lp = torch.where(there, lp, torch.zeros_like(lp))
    gain = lp.double() - s["ref"] if s["ref"] is not None else lp.double()
    total = torch.zeros(2 * c["pairs"], dtype=torch.float64, device="cuda")
    total.index_add_(0, seq[there], gain[there])
    reward = _BETA * total
    m = reward[0::2] - reward[1::2]
    small = torch.log(1 + torch.exp(-m.abs()))
    loss = (1 - c["eps"]) * (small - m.clamp(max=0)) + c["eps"] * (small + m.clamp(min=0))
    slope = c["eps"] - 1 / (1 + torch.exp(m))          # d loss / d m
    slope = torch.stack([slope, -slope], 1).flatten() * _BETA * s["scale"]
    slope = slope[seq.clamp(max=2 * c["pairs"] - 1)].float()
    return {"loss": loss.float(), "reward": reward.float(), "logp": lp, "d_logits": _to_logits(p, y, there, slope, dtype)}


# -- what a pass cannot do without ------------------------------------------------


def work(case):
    c = case
    t, v = c["tokens"], c["vocab"]
    live = t * (1.0 - c["pad"])              # rows that have to be read
    small = t * {"logp": 16, "logp_grad": 12, "distill": 12, "policy": 28, "pref": 16}[c["op"]]
    if c["op"] == "logp":
        return {"bytes": 2 * live * v + small, "flops": 4 * live * v}
    if c["op"] == "distill":
        small += t * c["top"] * (2 + c["ids"] // 8)
        sums = 2 if c["top"] and c["hard"] and c["temp"] != 1.0 else 1
        return {"bytes": 2 * (live + t) * v + small, "flops": (4 * sums + 4 * sums) * live * v}
    return {"bytes": 2 * (live + t) * v + small, "flops": 8 * live * v}


# -- the definitions in 64 bits ----------------------------------------------------


def _blocks(c):
    n = max(1, (1 << 26) // c["vocab"])
    return [slice(a, min(a + n, c["tokens"])) for a in range(0, c["tokens"], n)]


def _zeros(*shape):
    return torch.zeros(*shape, dtype=torch.float64, device="cuda")


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    op, temp = c["op"], c.get("temp", 1.0)
    live = torch.nonzero(s["targets"] >= 0).flatten()
    logp, lse = _zeros(c["tokens"]), _zeros(c["tokens"])
    for b in _blocks(c):
        x = s["logits"][b].double() / temp
        lse[b] = torch.logsumexp(x, dim=1)
        logp[b] = torch.log_softmax(x, dim=1)[torch.arange(x.shape[0], device="cuda"), s["targets"][b].clamp(min=0)]
    gone = torch.ones(c["tokens"], dtype=torch.bool, device="cuda")
    gone[live] = False
    logp[gone], lse[gone] = 0.0, 0.0
    if op == "logp":
        return {"logp": logp, "lse": lse}
    if op == "distill":
        loss, grad = _zeros(c["tokens"]), _zeros(c["tokens"], c["vocab"])
        for b in _blocks(c):
            n = s["logits"][b].shape[0]
            row = torch.arange(n, device="cuda")
            z = s["logits"][b].double()
            if c["top"]:
                ids = s["top_ids"][b].long()
                taught = s["top"][b].double() / temp
                q = torch.where(ids >= 0, torch.exp(taught - taught.amax(1, keepdim=True)), _zeros(1))
                q = q / q.sum(1, keepdim=True)
                lp = torch.log_softmax(z / temp, 1)
                at = torch.gather(lp, 1, ids.clamp(min=0))
                terms = torch.special.xlogy(q, q) - torch.where(q > 0, q * at, _zeros(1))
                loss[b] += c["soft"] * temp * temp * terms.sum(1)
                dense = _zeros(n, c["vocab"])
                dense.scatter_add_(1, ids.clamp(min=0), q)
                grad[b] += c["soft"] * temp * (lp.exp() - dense)
            if c["hard"]:
                lp = torch.log_softmax(z, 1)
                y = s["targets"][b].clamp(min=0)
                loss[b] -= c["hard"] * lp[row, y]
                p = lp.exp()
                p[row, y] = torch.expm1(lp[row, y])
                grad[b] += c["hard"] * p
        loss[gone], grad[gone] = 0.0, 0.0
        return {"loss": loss, "d_logits": grad * s["scale"]}
    out = {}
    if op == "logp_grad":
        slope = s["d_logp"].double()
    elif op == "policy":
        a, move, d = s["advantage"].double(), logp - s["old"].double(), s["ref"].double() - logp
        w = s["weight"].double() if s["weight"] is not None else torch.ones_like(a)
        inside = torch.where(a > 0, move <= math.log1p(_HIGH), move >= math.log1p(-_LOW))
        limit = torch.where(a > 0, 1 + _HIGH, 1 - _LOW) * a
        r = torch.exp(move)
        loss = w * (c["kl"] * (torch.expm1(d) - d) - torch.where(inside, r * a, limit))
        loss[gone] = 0.0
        slope = s["scale"] * w * (-c["kl"] * torch.expm1(d) - torch.where(inside, r * a, _zeros(1)))
        out = {"loss": loss, "logp": logp}
    else:
        starts = s["starts"].tolist()
        logp[starts[-1]:] = 0.0
        gain = logp - s["ref"].double() if s["ref"] is not None else logp.clone()
        gain[gone] = 0.0
        reward = _BETA * torch.stack([gain[a:b].sum() for a, b in zip(starts, starts[1:])])
        m = reward[0::2] - reward[1::2]
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - c["eps"]) * ls(m) - c["eps"] * ls(-m)
        dm = -(1 - c["eps"]) * torch.sigmoid(-m) + c["eps"] * torch.sigmoid(m)
        slope = _zeros(c["tokens"])
        for i, (a, b) in enumerate(zip(starts, starts[1:])):
            slope[a:b] = (dm[i // 2] if i % 2 == 0 else -dm[i // 2]) * _BETA * s["scale"]
        out = {"loss": loss, "reward": reward, "logp": logp}
    slope[gone] = 0.0
    grad = _zeros(c["tokens"], c["vocab"])
    for b in _blocks(c):
        lp = torch.log_softmax(s["logits"][b].double() / temp, 1)
        row, y = torch.arange(lp.shape[0], device="cuda"), s["targets"][b].clamp(min=0)
        p = -lp.exp()
        p[row, y] = -torch.expm1(lp[row, y])
        grad[b] = p * (slope[b] / temp)[:, None]
    return {**out, "d_logits": grad}
