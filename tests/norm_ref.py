"""Plain 64-bit definitions of the heads' norm with its rotary position, and of its gradient, for the tests."""
from __future__ import annotations

import numpy as np

from tests import attn_ref as ref


def root(x, eps):
    """1 / sqrt(mean(x^2) + eps) of every head, [..., 1]."""
    return 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def norm_rotate(x, w, eps, pos, f, m, rot, layout):
    """R(pos) (x r w): x [.., heads, D], w [D] with the offset added."""
    return ref.rotate(x * root(x, eps) * w, pos, f, m, rot, layout)


def size(x, rot, layout, m):
    """What a turned element's error goes by: |a| + |b| of its pair times the factor, |x| elsewhere."""
    i = np.arange(rot // 2)
    i0, i1 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    s = np.abs(x)
    s[..., i0] = s[..., i1] = (np.abs(x[..., i0]) + np.abs(x[..., i1])) * m
    return s


def gradient(x, dy, w, eps, pos, f, m, rot, layout):
    """(dx, dw, sizes of the terms of dx, of dw)."""
    g = ref.rotate(dy, pos, f, m, rot, layout, transpose=True)
    gs = size(dy, rot, layout, m)
    r = root(x, eps)
    mean = lambda a: np.mean(a, -1, keepdims=True)  # noqa: E731
    dx = r * (w * g - r * r * x * mean(w * g * x))
    dxs = r * (np.abs(w) * gs + r * r * np.abs(x) * mean(np.abs(w * x) * gs))
    axes = tuple(range(x.ndim - 1))
    return dx, (g * x * r).sum(axes), dxs, (gs * np.abs(x) * r).sum(axes)
