"""The float64 forms that the GPU tests compare with, against differences and against differentiation."""
import torch

import plain64


def _attention(Q, K, V, balls):
    out = torch.zeros_like(V)
    for idx in balls:
        idx = idx[idx >= 0]
        if len(idx):
            q, k, v = (t[idx].transpose(0, 1) for t in (Q, K, V))
            o = torch.softmax(q @ k.transpose(1, 2) / Q.shape[2] ** 0.5, 2) @ v
            out = out.index_copy(0, idx, o.transpose(0, 1))
    return out


def _inputs(rows, H, d, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, H, d, generator=g, dtype=torch.float64) for _ in range(n)]


def test_attention_backward_against_differentiation():
    Q, K, V, dO = _inputs(11, 2, 32, 4)
    perm = torch.tensor([3, 1, 0, 2, 9, 8, -1, -1, 4, 10, 5, 7, 6, -1, -1, -1, -1, -1, -1, -1])
    balls = plain64.ball_rows(perm, 20, 4)
    x = [t.clone().requires_grad_(True) for t in (Q, K, V)]
    want = torch.autograd.grad((_attention(*x, balls) * dO).sum(), x)
    got, _ = plain64.attention_backward(Q, K, V, dO, balls)
    for a, b in zip(got, want):
        assert (a - b).abs().max() < 1e-13


def test_attention_backward_against_differences(orc):
    # central differences of the oracle's forward pass along random directions
    Q, K, V, dO = _inputs(12, 2, 32, 4, seed=1)
    perm = torch.tensor([0, 5, 2, 7, 11, 1, 3, 4, 6, 8, 9, 10], dtype=torch.int32)
    balls = plain64.ball_rows(perm, 12, 6)
    got, _ = plain64.attention_backward(Q, K, V, dO, balls)
    h = 1e-5
    for i in range(3):
        dirn = _inputs(12, 2, 32, 1, seed=5 + i)[0]

        def loss(t):
            x = [Q, K, V]
            x[i] = x[i] + t * dirn
            return float((_attention(*x, balls) * dO).sum())
        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - float((got[i] * dirn).sum())) < 1e-7 * max(1, abs(diff))
    # the same forward pass as the oracle's
    o = orc.ball_attention(*(t.float().numpy() for t in (Q, K, V)), 6, perm.numpy())
    assert abs(o - _attention(*(t.float().double() for t in (Q, K, V)), balls).numpy()).max() < 1e-9


def test_norm_backward_against_differentiation_and_differences():
    g = torch.Generator().manual_seed(3)
    h, dY, dH = (torch.randn(5, 7, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(7, generator=g, dtype=torch.float64)
    dx, dw, _, _ = plain64.rms_norm_backward(dY, h, w, dH, 1e-3)
    x, v = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    y = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-3) * v
    a, b = torch.autograd.grad((y * dY).sum() + (x * dH).sum(), (x, v))
    assert (a - dx).abs().max() < 1e-13 and (b - dw).abs().max() < 1e-13
    t = 1e-6
    dirn = torch.randn(5, 7, generator=g, dtype=torch.float64)
    f = [float((plain64.rms_norm(h + s * t * dirn, w, 1e-3)[0] * dY).sum() + ((h + s * t * dirn) * dH).sum())
         for s in (1, -1)]
    assert abs((f[0] - f[1]) / (2 * t) - float((dx * dirn).sum())) < 1e-7
