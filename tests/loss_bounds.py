"""Bounds on the gradients of the vocabulary loss, for the GPU tests.

bf16 keeps 8 bits: a rounding is off by at most half a unit in the last place,
2^-8 of the value, evenly spread and so 2^-8 / sqrt(3) of it in the root mean
square at most.

  fp32 outputs   G is held as the sum of two bf16 values, off by 2^-16 at most.
  bf16 outputs   G is rounded once, but not at the label (that rounding is added
                 to the sums again, itself to 2^-16): eight standard deviations of
                 the others' are allowed, and the output's own rounding.
  both           the logits are recomputed: 4 el (el: the largest error of a
                 logit, (d / 32 + 32) 2^-24 sum |h w|); a hardware exponential and
                 the fp32 sums: 2e-5 of the terms' sizes.
"""

import numpy as np

U = 2.0 ** -8


def logit_error(h, w):
    return (h.shape[1] / 32 + 32) * 2.0 ** -24 * float((np.abs(h) @ np.abs(w).T).max(initial=0))


def bounds(G, h, w, rows, labels, el, dh_dtype, dw_dtype):
    """Bounds, by element, on the errors of dh = G w and dw = G^T h; G, h, labels: the labelled tokens' (all of
    them finite), ``rows`` = arange(len(labels))."""
    rest = G.copy()
    rest[rows, labels] = 0
    out = []
    for g, r, b, dt in ((G, rest, w, dh_dtype), (G.T, rest.T, h, dw_dtype)):
        ref, size = np.abs(g @ b), np.abs(g) @ np.abs(b)
        tol = (4 * el + 2e-5 + U * U) * size
        if dt == "bf16":
            tol += 8 * U / 3 ** 0.5 * np.sqrt((r * r) @ (b * b))
            tol += U * (ref + tol)
        else:
            tol += 2.0 ** -23 * ref
        out.append(tol + 1e-30)
    return out


def bf16(x):
    """Rounded to bf16 (nearest even), as float64."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7fff + ((b >> 16) & 1)) & np.uint32(0xffff0000)).view(np.float32).astype(np.float64)
