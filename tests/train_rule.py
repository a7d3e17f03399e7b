"""Which instance of a kernel the norm and the table gradient choose for a size:
their rules (norm_shape in zero_norm.cu, grad_space in zero_embed.cu) written
again, so that tests can say which instances their sizes run."""
from __future__ import annotations

SMS = 152


def up(n, m):
    return -(-n // m) * m


def norm(rows, cols, backward):
    """(vectors a thread, wide, the vectors cover the row exactly), rows a CTA, and whether a
    CTA takes more rows than it holds at a time."""
    nv = -(-cols // 8)
    v = 1 if nv <= 512 else 4
    if rows >= 608 and nv >= 64:
        v = 2 if nv < 128 or (backward and nv <= 512) else 4
    g = up(-(-nv // v), 32)
    per = 1 if g >= 128 else 128 // g
    wide = v == 4 and g > 256
    full = v > 1 and not wide and g * v * 8 == cols
    most = 1024 if v == 1 or wide else (2 if backward else 3) * 256
    ctas = min(-(-rows // per), SMS * max(1, most // (g * per)))
    if backward:
        ctas = min(ctas, 1216)
    return (v, wide, full), per, ctas * per < rows


def norm_workspace(rows, cols):
    _, per, _ = norm(rows, cols, True)
    return min(-(-rows // per), 1216) * up(cols, 8) * 4


def cells_per_cta(slots, cell):
    fit = 256 // slots if slots < 256 else 1
    return min(fit, 1024 // cell)


def table_layout(tokens, dim):
    if tokens > 20000:
        return "many"
    wide = cells_per_cta(-(-dim // 8), 16) * 16
    return "some" if -(-tokens // wide) > 456 else "few"


def table_workspace(tokens, dim):
    """Up to 65,536 tokens: the pairs and two partial rows a cell."""
    cell = 32 if table_layout(tokens, dim) == "many" else 16
    return up(8 * tokens, 256) + -(-tokens // cell) * -(-dim // 8) * 64
