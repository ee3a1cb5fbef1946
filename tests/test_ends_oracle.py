"""Pins for oracle/ends_oracle.py: hand-worked values, torch autograd in fp64,
central differences, and torch's own clipping."""

import numpy as np
import torch

from oracle import ends_oracle as A


def test_embed_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    x = A.embed(table, [2, -1, 0, 3], 2.0)
    assert np.array_equal(x, [[10.0, 12.0], [0.0, 0.0], [2.0, 4.0], [0.0, 0.0]])
    dx = np.array([[1.0, 2.0], [9.0, 9.0], [4.0, 8.0], [9.0, 9.0], [0.5, 0.25]])
    g = A.embed_backward(dx, [2, -1, 0, 3, 2], 3, 2.0)
    assert np.array_equal(g, [[8.0, 16.0], [0.0, 0.0], [3.0, 4.5]])
    assert np.array_equal(A.embed_backward(dx[:1], [1], 3, 1.0, base=np.ones((3, 2))), [[1, 1], [2, 3], [1, 1]])


def test_embed_backward_is_autograd_and_differences():
    r = np.random.default_rng(0)
    V, d, T = 7, 5, 30
    table, dx = r.standard_normal((V, d)), r.standard_normal((T, d))
    tokens = r.integers(0, V, T)
    w = torch.tensor(table, requires_grad=True)
    (torch.nn.functional.embedding(torch.tensor(tokens), w) * 1.5 * torch.tensor(dx)).sum().backward()
    g = A.embed_backward(dx, tokens, V, 1.5)
    assert np.allclose(g, w.grad.numpy(), rtol=1e-13, atol=1e-13)
    v = r.standard_normal((V, d))
    f = lambda h: (A.embed(table + h * v, tokens, 1.5) * dx).sum()  # noqa: E731
    assert np.isclose((f(1e-3) - f(-1e-3)) / 2e-3, (g * v).sum(), rtol=1e-9)


def test_clip_by_hand_and_as_torch_does():
    norm, out = A.clip([np.array([3.0]), np.array([[0.0, 4.0]])], 2.5)
    assert norm == 5.0 and np.array_equal(out[0], [1.5]) and np.array_equal(out[1], [[0.0, 2.0]])
    norm, out = A.clip([np.array([3.0]), np.array([4.0])], 5.0)
    assert norm == 5.0 and out[0][0] == 3.0
    norm, out = A.clip([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and out[0][1] == 1.0
    r = np.random.default_rng(1)
    gs = [r.standard_normal(s) for s in ((3, 4), (5,), (2, 2, 2))]
    ps = [torch.zeros(g.shape, dtype=torch.float64, requires_grad=True) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.tensor(g)
    tn = torch.nn.utils.clip_grad_norm_(ps, 0.7)
    norm, out = A.clip(gs, 0.7)
    assert np.isclose(norm, float(tn), rtol=1e-12)
    for p, o in zip(ps, out):   # torch divides by norm + 1e-6
        assert np.allclose(p.grad.numpy(), o, rtol=2e-6)
