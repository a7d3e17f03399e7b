"""How the losses' rows are laid on the GPU for a size: the rule (layout_of in
zero_loss.cuh) written again, so that tests can say which instances their sizes
run."""
from __future__ import annotations

SMS = 152


def chunk(vecs, ctas):
    return -(-(-(-vecs // ctas)) // 8) * 8


def layout(rows, vocab, grad=True, top=False):
    """(threads of a CTA, CTAs of a row)"""
    vecs = -(-vocab // 8)
    ctas, fit, best = 8, 2, 0.0
    for c in range(1, 9):
        size = 16 * (chunk(vecs, c) + 8) + 6 * 1024
        n = min(228 * 1024 // size, 4)
        fill = n * size / (1.0 + (0.1 if grad and not top else 0.05) * (c - 1))
        if n >= (2 if grad else 3) and fill > best:
            best, ctas, fit = fill, c, n
        if n >= 4:
            break
    if rows <= 4 * SMS:
        while 2 * ctas <= 8 and 2 * ctas * rows <= SMS and chunk(vecs, ctas) > 512:
            ctas *= 2
        c = chunk(vecs, ctas)
        return (32 if vecs <= 64 else 128 if c <= 512 else 256 if ctas > 1 else 512), ctas
    return (32 if vecs <= 512 else 128 if vecs <= 1024 or not grad else 512 if fit == 2 and not top else 256), ctas
