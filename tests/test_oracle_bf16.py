"""The FP64 oracle of the bf16 GroupedLinear's gradients and of the adapter linear:
against central differences, loops and an independent torch formulation."""
import numpy as np
import torch

from oracle import bf16_oracle as B

RNG = np.random.default_rng(5)
OFF = np.array([0, 3, 3, 4, 9])


def case(r=True):
    M, K, N, E = 9, 5, 4, 4
    return (RNG.standard_normal((M, N)), RNG.standard_normal((M, K)), RNG.standard_normal((E, N, K)),
            RNG.random(M) if r else None)


def test_gradients_against_differences():
    dy, x, w, r = case()
    dx, dw, dr = B.linear_bwd(dy, x, w, OFF, r)
    loss = lambda: float((B.linear_fwd(x, w, OFF, r) * dy).sum())
    h = 1e-4
    for t, g in ((x, dx), (w, dw), (r, dr)):
        num = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            old = t[i]
            t[i] = old + h
            up = loss()
            t[i] = old - h
            num[i] = (up - loss()) / (2 * h)
            t[i] = old
        # the loss is linear in each value: differences are exact up to rounding
        assert np.abs(num - g).max() < 1e-9


def test_gradients_against_autograd():
    for scaled in (False, True):
        dy, x, w, r = case(scaled)
        tx, tw = (torch.tensor(t, requires_grad=True) for t in (x, w))
        tr = None if r is None else torch.tensor(r, requires_grad=True)
        y = torch.cat([tx[OFF[e]:OFF[e + 1]] @ tw[e].T for e in range(4)])
        y = y if tr is None else y * tr[:, None]
        y.backward(torch.tensor(dy))
        dx, dw, dr = B.linear_bwd(dy, x, w, OFF, r)
        assert np.allclose(dx, tx.grad, rtol=0, atol=1e-12)
        assert np.allclose(dw, tw.grad, rtol=0, atol=1e-12)
        assert (dr is None) if r is None else np.allclose(dr, tr.grad, rtol=0, atol=1e-12)
        assert not dw[1].any()


def test_adapters_against_a_merged_weight():
    M, K, N, r, L = 7, 6, 5, 3, 2
    x, w = RNG.standard_normal((M, K)), RNG.standard_normal((N, K))
    a, b = RNG.standard_normal((L, r, K)), RNG.standard_normal((L, N, r))
    ids, s = np.array([0, 1, -1, 1, 2, 0, -7]), np.array([0.5, 2.0])
    y = B.lora_fwd(x, w, a, b, ids, s)
    for m, l in enumerate(ids):
        merged = w + (s[l] * b[l] @ a[l] if 0 <= l < L else 0)
        assert np.allclose(y[m], merged @ x[m], rtol=0, atol=1e-12)
    assert np.allclose(B.lora_fwd(x, w, a, b, np.full(M, -1)), x @ w.T)
    assert (B.lora_bound(x, w, a, b, ids, s) > 0).all()
