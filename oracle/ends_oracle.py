"""CPU oracle for a model's two ends: the embedding with its gradient, and the
global norm of the gradients with clipping.  TEST INFRASTRUCTURE ONLY; fp64
NumPy, no code shared with the GPU library.

    embed   x_t = scale table[token_t]; zeros for a token outside [0, V)
    dtable  dtable_v = scale sum_{t: token_t = v} dx_t
    clip    norm = sqrt(sum of squares); g min(1, max_norm / norm), g where the norm is not finite
"""

from __future__ import annotations

import numpy as np

F64 = np.float64


def embed(table, tokens, scale: float) -> np.ndarray:
    V, d = table.shape
    x = np.zeros((len(tokens), d), F64)
    for t, v in enumerate(tokens):
        if 0 <= v < V:
            x[t] = scale * np.asarray(table[v], F64)
    return x


def embed_backward(dx, tokens, V: int, scale: float, base=None) -> np.ndarray:
    """The gradient, on top of ``base`` where given."""
    out = np.zeros((V, dx.shape[1]), F64) if base is None else np.array(base, F64)
    for t, v in enumerate(tokens):
        if 0 <= v < V:
            out[v] += scale * np.asarray(dx[t], F64)
    return out


def embed_magnitude(dx, tokens, V: int, scale: float, base=None) -> np.ndarray:
    """The sizes of the terms of embed_backward, summed: what its rounding errors are relative to."""
    return embed_backward(np.abs(dx), tokens, V, abs(scale), None if base is None else np.abs(base))


def sumsq(grads) -> float:
    return float(sum((np.asarray(g, F64) ** 2).sum() for g in grads))


def clip(grads, max_norm: float):
    """(norm, clipped gradients)."""
    norm = np.sqrt(sumsq(grads))
    f = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, [np.asarray(g, F64) * f for g in grads]
