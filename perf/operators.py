"""Workloads of the training operators next to the sharded optimizer step.

The optimizer step reads 16-bit gradient rows and writes 16-bit parameters.
The operators here are what stands between the two in a language model's
training: the embedding lookup and its gradient, the residual addition with
the root-mean-square norm and its gradient, and activation checkpoints in 8
bits, which the norm writes and the backward pass reads (the norm's gradient
and the weight gradient of the linear layer behind it).

Every case names its operator in ``"op"``; ``run`` does one pass of it, either
in plain torch operations in 32 bits or through the framework's entry points
(``own``).

The 8-bit checkpoint of a [rows, cols] matrix holds, for every block of 32
consecutive elements of a row, one byte s and 32 signed bytes q that stand for
q * 2**(s - 127).  With a the block's largest magnitude, k = s - 127 is the
smallest integer with a <= 127 * 2**k, kept inside the limits of the
activations' type (f16: -24..9, bf16: -127..121), and q = rint(x / 2**k) kept
inside -127..127.  A block holding an inf or NaN has s = 255 and stands for NaN.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_LIMITS = {"f16": (-24, 9), "bf16": (-127, 121)}
_EPS = 1e-5
_BLOCK = 32


def listed():
    return [
        # One token of a decoding or probing loop: what it costs is latency.
        dict(name="lookup_token", op="lookup", tokens=1, vocab=50257, dim=768, dtype="bf16", scale=1.0, pad=0.0),
        # A training micro-batch of the 1.5B model's width, embeddings scaled by sqrt(dim).
        dict(name="lookup_batch", op="lookup", tokens=32768, vocab=50257, dim=1600, dtype="f16", scale=40.0, pad=0.0),
        # A short, odd batch with padding, added onto the gradient that a tied output layer left in the row.
        dict(name="egrad_tied", op="egrad", tokens=1021, vocab=50257, dim=768, dtype="bf16", scale=1.0, pad=0.06, add=True),
        # The whole table's gradient of a long batch: frequent tokens take thousands of rows, most of the table none.
        dict(name="egrad_batch", op="egrad", tokens=65536, vocab=50257, dim=1600, dtype="f16", scale=40.0, pad=0.0, add=False),
        # Serving: residual and norm of a single token, nothing kept for a backward pass.
        dict(name="norm_token", op="norm", rows=1, cols=1600, dtype="f16", gain=True, residual=True),
        # A training micro-batch: forward with its checkpoint, then backward from it.
        dict(name="norm_train", op="norm_train", rows=16384, cols=4096, dtype="bf16", gain=True, residual=True, add=False),
        # Backward alone with odd sizes, no residual branch, gain gradient added over micro-batches.
        dict(name="norm_back_odd", op="norm_back", rows=2047, cols=1601, dtype="f16", gain=True, residual=False, add=True),
        # The 8-bit checkpoint of a hidden layer's activations, written and read back (4 x 1600 wide).
        dict(name="ckpt_batch", op="ckpt", rows=16384, cols=6400, dtype="bf16"),
        # The same, few odd rows.
        dict(name="ckpt_odd", op="ckpt", rows=333, cols=1111, dtype="f16"),
        # Weight gradient of an attention projection of the 1.5B model: few output tiles, a long sum.
        dict(name="wgrad_proj", op="wgrad", tokens=4096, cols=1600, outs=1600, dtype="f16", gain=True, add=True),
        # A ragged head of the same width on an odd number of tokens.
        dict(name="wgrad_odd", op="wgrad", tokens=2049, cols=768, outs=1001, dtype="bf16", gain=False, add=False),
        # The expanding layer of a 4096-wide model on a long micro-batch: the matrix product alone counts.
        dict(name="wgrad_wide", op="wgrad", tokens=16384, cols=4096, outs=16384, dtype="bf16", gain=True, add=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd about as often as even."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def _width(rng, lo, hi):
    """A matrix width: a multiple of 64, or any."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.6:
        n = max(64, n // 64 * 64)
    return n + 64 if n == 3072 else n


def draw(rng):
    op = rng.choice(["lookup", "egrad", "norm", "norm_train", "norm_back", "ckpt", "wgrad"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("lookup", "egrad"):
        c = dict(op=op, tokens=_log(rng, 1, 65536), vocab=_log(rng, 1000, 131072), dim=_width(rng, 64, 2048), dtype=dtype,
                 scale=rng.choice([1.0, 40.0]), pad=rng.choice([0.0, 0.1]))
        if op == "egrad":
            c["add"] = rng.random() < 0.5
        return c
    if op in ("norm", "norm_train", "norm_back"):
        c = dict(op=op, rows=_log(rng, 1, 16384), cols=_width(rng, 64, 8192), dtype=dtype, gain=rng.random() < 0.8,
                 residual=rng.random() < 0.7)
        if op != "norm":
            c["add"] = rng.random() < 0.5
        return c
    if op == "ckpt":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_width(rng, 64, 8192), dtype=dtype)
    return dict(op=op, tokens=_log(rng, 1, 16384), cols=_width(rng, 64, 4096), outs=_width(rng, 64, 8192), dtype=dtype,
                gain=rng.random() < 0.5, add=rng.random() < 0.5)


# -- inputs --------------------------------------------------------------------


def _up(n, m):
    return -(-n // m) * m


def _matrix(rows, cols, dtype):
    """An activation matrix whose rows start on 16-byte boundaries, as the framework lays its rows out."""
    return torch.empty(rows, _up(cols, 8), dtype=dtype, device="cuda")[:, :cols]


def _normal(g, rows, cols, dtype, sigma, channels=0.0):
    """Normal values; some channels `channels` times larger, as residual streams have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * sigma
    if channels:
        x[:, 5::97] *= channels
    out = _matrix(rows, cols, dtype)
    out.copy_(x)
    return out


def _ids(g, tokens, vocab, pad):
    """Token numbers: frequency falls as 1 / (number + 1), as vocabularies sorted by frequency have it; `pad` of them are
    padding (-1)."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(vocab)).long().clamp(1, vocab) - 1
    if pad:
        ids[torch.rand(tokens, generator=g, device="cuda") < pad] = -1
    return ids


def _ckpt_of(x, dtype):
    """The checkpoint of x in its stored form: q [rows, pitch] int8 and s [rows, blocks] uint8."""
    k, q, bad = _quantise(x.float(), dtype)
    rows, blocks, _ = q.shape
    store = torch.zeros(rows, _up(blocks * _BLOCK, 16), dtype=torch.int8, device="cuda")
    store[:, : blocks * _BLOCK] = q.reshape(rows, -1).to(torch.int8)
    s = torch.where(bad, torch.full_like(k, 255), k + 127).to(torch.uint8)
    return store[:, : x.shape[1]], s.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    op, dtype = c["op"], _TYPES[c["dtype"]]
    s = {"case": c}
    grad_sigma = 1e-3 * (1024.0 if c["dtype"] == "f16" else 1.0)   # f16 gradients are loss-scaled
    if op in ("lookup", "egrad"):
        s["ids"] = _ids(g, c["tokens"], c["vocab"], c["pad"])
        if op == "lookup":
            s["table"] = (torch.randn(c["vocab"], c["dim"], generator=g, device="cuda") * 0.02).to(dtype)
        else:
            s["d_out"] = _normal(g, c["tokens"], c["dim"], dtype, grad_sigma)
            old = torch.randn(c["vocab"], c["dim"], generator=g, device="cuda") * grad_sigma if c["add"] else \
                torch.zeros(c["vocab"], c["dim"], device="cuda")
            s["d_table"] = old.to(dtype)
    elif op in ("norm", "norm_train", "norm_back"):
        rows, cols = c["rows"], c["cols"]
        s["gain"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dtype) if c["gain"] else None
        if op != "norm_back":
            s["x"] = _normal(g, rows, cols, dtype, 0.5)
            s["res"] = _normal(g, rows, cols, dtype, 2.0, 12.0) if c["residual"] else None
        if op != "norm":
            s["dy"] = _normal(g, rows, cols, dtype, grad_sigma)
            s["d_res"] = _normal(g, rows, cols, dtype, grad_sigma) if c["residual"] else None
            old = torch.randn(cols, generator=g, device="cuda") * grad_sigma if c["add"] else torch.zeros(cols, device="cuda")
            s["d_gain"] = old.to(dtype)
        if op == "norm_back":
            h = _normal(g, rows, cols, dtype, 2.0, 12.0).float()
            s["rstd"] = torch.rsqrt((h * h).mean(-1) + _EPS)
            s["q"], s["s"] = _ckpt_of(h * s["rstd"][:, None], c["dtype"])
    elif op == "ckpt":
        s["x"] = _normal(g, c["rows"], c["cols"], dtype, 1.0, 12.0)
    else:
        s["dy"] = _normal(g, c["tokens"], c["outs"], dtype, grad_sigma)
        s["q"], s["s"] = _ckpt_of(_normal(g, c["tokens"], c["cols"], torch.float32, 1.0, 8.0), c["dtype"])
        s["gain"] = (1.0 + 0.2 * torch.randn(c["cols"], generator=g, device="cuda")).to(dtype) if c["gain"] else None
        old = torch.randn(c["outs"], c["cols"], generator=g, device="cuda") * grad_sigma if c["add"] else \
            torch.zeros(c["outs"], c["cols"], device="cuda")
        s["dw"] = old.to(dtype)
    if own:
        s["call"] = _handles(s, c, op, dtype)
    return s


def _handles(s, c, op, dtype):
    """What a user's program sets up once for its buffers: the output buffers and workspaces, and the descriptors of the
    buffers that it passes with every step."""
    import zero_sharded_optimizer_02_gb300 as z
    h = {"z": z}
    space = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
    if op in ("lookup", "egrad"):
        h["ids"] = z.ids(s["ids"])
        h["flag"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "lookup":
            s["out"] = _matrix(c["tokens"], c["dim"], dtype)
            h["table"], h["out"] = z.mat(s["table"]), z.mat(s["out"])
        else:
            h["d_out"], h["d_table"] = z.mat(s["d_out"]), z.mat(s["d_table"])
            h["ws"] = space(z.zero_embed_grad_workspace(c["tokens"], c["vocab"], c["dim"]))
        return h
    if op in ("norm", "norm_train", "norm_back"):
        rows, cols = c["rows"], c["cols"]
        if op != "norm_back":
            s["h"], s["y"] = _matrix(rows, cols, dtype), _matrix(rows, cols, dtype)
            h["x"], h["h"], h["y"] = z.mat(s["x"]), z.mat(s["h"]), z.mat(s["y"])
            h["res"] = z.mat(s["res"]) if s["res"] is not None else None
            s["rstd"] = torch.empty(rows, device="cuda")
        if op == "norm_train":
            s["q"], s["s"] = z.act8_empty(rows, cols)
        if op != "norm":
            s["dx"] = _matrix(rows, cols, dtype)
            h["ckpt"] = z.act8(s["q"], s["s"])
            h["dy"], h["dx"] = z.mat(s["dy"]), z.mat(s["dx"])
            h["d_res"] = z.mat(s["d_res"]) if s["d_res"] is not None else None
            h["ws"] = space(z.zero_norm_backward_workspace(rows, cols))
        return h
    if op == "ckpt":
        s["q"], s["s"] = z.act8_empty(c["rows"], c["cols"])
        s["out"] = _matrix(c["rows"], c["cols"], dtype)
        h["ckpt"], h["x"], h["out"] = z.act8(s["q"], s["s"]), z.mat(s["x"]), z.mat(s["out"])
        return h
    h["ckpt"], h["dy"], h["dw"] = z.act8(s["q"], s["s"]), z.mat(s["dy"]), z.mat(s["dw"])
    h["ws"] = space(z.zero_act_weight_grad_workspace(c["tokens"], c["outs"], c["cols"]))
    return h


# -- one pass ------------------------------------------------------------------


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c, h = s["case"], s["call"]
    z, op = h["z"], c["op"]
    if op == "lookup":
        z.zero_embed_lookup(h["table"], h["ids"], c["scale"], h["out"], h["flag"])
        return {"out": s["out"]}
    if op == "egrad":
        z.zero_embed_grad(h["d_out"], h["ids"], c["scale"], c["add"], h["d_table"], h["ws"], h["ws"].numel(), h["flag"])
        return {"d_table": s["d_table"]}
    if op == "norm":
        z.zero_norm_forward(h["x"], h["res"], s["gain"], _EPS, h["h"], h["y"], None, None)
        return {"h": s["h"], "y": s["y"]}
    if op == "norm_train":
        z.zero_norm_forward(h["x"], h["res"], s["gain"], _EPS, h["h"], h["y"], s["rstd"], h["ckpt"])
    if op in ("norm_train", "norm_back"):
        z.zero_norm_backward(h["dy"], h["ckpt"], s["rstd"], s["gain"], h["d_res"], h["dx"], s["d_gain"], c["add"], h["ws"],
                             h["ws"].numel())
        out = {"dx": s["dx"], "d_gain": s["d_gain"]}
        return {**out, "h": s["h"], "y": s["y"], "rstd": s["rstd"]} if op == "norm_train" else out
    if op == "ckpt":
        z.zero_act_pack(h["x"], h["ckpt"])
        z.zero_act_unpack(h["ckpt"], h["out"])
        return {"out": s["out"]}
    z.zero_act_weight_grad(h["dy"], h["ckpt"], s["gain"], c["add"], h["dw"], h["ws"], h["ws"].numel())
    return {"dw": s["dw"]}


def _power(k):
    """2**k in 32 bits for whole k in -127..127, exact (an exponential function need not be)."""
    return torch.where(k > -127, (k + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, dtype):
    """(k, q, bad) of x in 32 bits, in blocks: the step's exponent, the whole numbers and whether the block is not finite."""
    lo, hi = _LIMITS[dtype]
    rows, cols = x.shape
    blocks = -(-cols // _BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * _BLOCK - cols)).view(rows, blocks, _BLOCK)
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    m, e = torch.frexp(torch.where(bad, torch.zeros_like(a), a))   # a = m * 2**e, 0.5 <= m < 1
    k = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(lo, hi)
    k = torch.where(m == 0, torch.full_like(k, lo), k)
    q = torch.round(x * _power(-k)[..., None]).clamp(-127, 127)
    return k, torch.where(bad[..., None], torch.zeros_like(q), q), bad


def _stands_for(k, q, bad, cols):
    """The values that a checkpoint stands for, in 32 bits."""
    v = q * _power(k)[..., None]
    v = torch.where(bad[..., None], torch.full_like(v, math.nan), v)
    return v.reshape(v.shape[0], -1)[:, :cols]


def _stored_values(q, s):
    """The values of a stored checkpoint, in 32 bits."""
    step = _power(torch.where(s == 255, 127, s.int() - 127))
    step = torch.where(s == 255, torch.full_like(step, math.nan), step)
    return q.float() * step.repeat_interleave(_BLOCK, dim=1)[:, : q.shape[1]]


def _norm_back(s, xhat, rstd, dtype):
    dy = s["dy"].float()
    u = dy * s["gain"].float() if s["gain"] is not None else dy
    dx = rstd[:, None] * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    if s["d_res"] is not None:
        dx = dx + s["d_res"].float()
    d_gain = (dy * xhat).sum(0)
    if s["case"]["add"]:
        d_gain = d_gain + s["d_gain"].float()
    s["d_gain"].copy_(d_gain)
    return {"dx": dx.to(dtype), "d_gain": s["d_gain"]}


def _run_plain(s):
    c = s["case"]
    op, dtype = c["op"], _TYPES[c["dtype"]]
    if op == "lookup":
        there = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        out = s["table"][s["ids"].clamp(0, c["vocab"] - 1)].float() * c["scale"]
        return {"out": torch.where(there[:, None], out, torch.zeros_like(out)).to(dtype)}
    if op == "egrad":
        there = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        rows = torch.where(there[:, None], s["d_out"].float(), torch.zeros((), device="cuda"))
        total = torch.zeros(c["vocab"], c["dim"], device="cuda")
        total.index_add_(0, s["ids"].clamp(0, c["vocab"] - 1), rows)
        total = total * c["scale"]
        if c["add"]:
            total = total + s["d_table"].float()
        s["d_table"].copy_(total)
        return {"d_table": s["d_table"]}
    if op in ("norm", "norm_train"):
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        rstd = torch.rsqrt((h * h).mean(-1) + _EPS)
        xhat = h * rstd[:, None]
        y = (xhat * s["gain"].float() if s["gain"] is not None else xhat).to(dtype)
        out = {"h": h.to(dtype), "y": y}
        if op == "norm":
            return out
        kept = _stands_for(*_quantise(xhat, c["dtype"]), c["cols"])
        return {**out, "rstd": rstd, **_norm_back(s, kept, rstd, dtype)}
    if op == "norm_back":
        return _norm_back(s, _stored_values(s["q"], s["s"]), s["rstd"], dtype)
    if op == "ckpt":
        return {"out": _stands_for(*_quantise(s["x"].float(), c["dtype"]), c["cols"]).to(dtype)}
    dw = s["dy"].float().t() @ _stored_values(s["q"], s["s"])
    if s["gain"] is not None:
        dw = dw * s["gain"].float()
    if c["add"]:
        dw = dw + s["dw"].float()
    s["dw"].copy_(dw)
    return {"dw": s["dw"]}


# -- what a pass cannot do without ------------------------------------------------


def _rows_met(c):
    """How many different tokens a batch holds, as its distribution has it."""
    edge = torch.log(torch.arange(1, c["vocab"] + 1, dtype=torch.float64)) / math.log(c["vocab"])
    share = (edge[1:] - edge[:-1]) * (1.0 - c["pad"])
    return float((1.0 - (1.0 - share) ** c["tokens"]).sum())


def work(case):
    c = case
    op = c["op"]
    if op == "lookup":
        moved = c["tokens"] * c["dim"]
        return {"bytes": 2 * moved + 2 * _rows_met(c) * c["dim"] + 8 * c["tokens"], "flops": moved}
    if op == "egrad":
        read = c["tokens"] * c["dim"] * (1.0 - c["pad"])
        rows = _rows_met(c)   # an added gradient leaves the other rows alone
        table = 4 * rows * c["dim"] if c["add"] else 2 * c["vocab"] * c["dim"]
        return {"bytes": 2 * read + 8 * c["tokens"] + table, "flops": read}
    if op in ("norm", "norm_train", "norm_back"):
        n = c["rows"] * c["cols"]
        kept = n + c["rows"] * -(-c["cols"] // _BLOCK) + 4 * c["rows"]
        forward = n * (6 + 2 * c["residual"]) + 2 * c["cols"] * c["gain"]
        if op == "norm":
            return {"bytes": forward, "flops": 5 * n}
        back = n * (4 + 2 * c["residual"]) + 2 * c["cols"] * (1 + c["gain"] + c["add"]) + kept
        if op == "norm_back":
            return {"bytes": back, "flops": 10 * n}
        return {"bytes": forward + kept + back, "flops": 19 * n}
    if op == "ckpt":
        n = c["rows"] * c["cols"]
        return {"bytes": 4 * n + 2 * (n + c["rows"] * -(-c["cols"] // _BLOCK)), "flops": 4 * n}
    t, o, i = c["tokens"], c["outs"], c["cols"]
    return {"bytes": 2 * t * o + t * i + t * -(-i // _BLOCK) + 2 * o * i * (1 + c["add"]) + 2 * i * c["gain"],
            "flops": 2 * t * o * i}


# -- the definitions in 64 bits ----------------------------------------------------


def _two_to(k):
    """2**k in 64 bits for whole k, exact."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _kept64(x, dtype):
    """The values that the checkpoint of x (64 bits) stands for: the step found by comparison, block by block."""
    lo, hi = _LIMITS[dtype]
    out = torch.empty_like(x)
    for b in range(0, x.shape[1], _BLOCK):
        block = x[:, b: b + _BLOCK]
        a = block.abs().amax(1, keepdim=True)
        k = torch.ceil(torch.log2((a / 127.0).clamp_min(2.0 ** -200)))
        k = torch.where(127.0 * _two_to(k - 1) >= a, k - 1, k)       # the logarithm may be off by a rounding
        k = torch.where(127.0 * _two_to(k) < a, k + 1, k).clamp(lo, hi)
        out[:, b: b + _BLOCK] = (block / _two_to(k)).round().clamp(-127, 127) * _two_to(k)
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    op = c["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    one = torch.ones((), dtype=torch.float64, device="cuda")
    if "q" in s:
        step = _two_to(s["s"].long() - 127)
        kept = s["q"].double() * step[:, torch.arange(c["cols"], device="cuda") // _BLOCK]
    if op == "lookup":
        out = torch.zeros(c["tokens"], c["dim"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0).flatten()
        out[at] = c["scale"] * d["table"][s["ids"][at]]
        return {"out": out}
    if op == "egrad":
        order = torch.argsort(s["ids"])
        order = order[s["ids"][order] >= 0]
        rows, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
        sums = torch.segment_reduce(d["d_out"][order].contiguous(), "sum", lengths=counts) if len(order) else \
            torch.zeros(0, c["dim"], dtype=torch.float64, device="cuda")
        total = d["d_table"].clone() if c["add"] else torch.zeros_like(d["d_table"])
        total[rows] += c["scale"] * sums
        return {"d_table": total}
    if op in ("norm", "norm_train", "norm_back"):
        gain = d["gain"] if c["gain"] else one
        out = {}
        if op == "norm_back":
            rstd = d["rstd"]
        else:
            h = d["x"] + d["res"] if c["residual"] else d["x"]
            rstd = 1.0 / torch.sqrt((h ** 2).sum(1) / c["cols"] + _EPS)
            out = {"h": h, "y": h * rstd.unsqueeze(1) * gain}
        if op == "norm":
            return out
        if op == "norm_train":
            kept = _kept64(h * rstd.unsqueeze(1), c["dtype"])
            out["rstd"] = rstd
        inner = (d["dy"] * gain * kept).sum(1, keepdim=True) / c["cols"]
        dx = (d["dy"] * gain - kept * inner) * rstd.unsqueeze(1)
        out["dx"] = dx + d["d_res"] if c["residual"] else dx
        out["d_gain"] = torch.einsum("tc,tc->c", d["dy"], kept) + (d["d_gain"] if c["add"] else 0.0)
        return out
    if op == "ckpt":
        return {"out": _kept64(d["x"], c["dtype"])}
    dw = torch.einsum("to,ti->oi", d["dy"], kept)
    dw = dw * (d["gain"] if c["gain"] else one)
    return {"dw": dw + d["dw"] if c["add"] else dw}
