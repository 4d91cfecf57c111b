"""Plain float64 forms (torch, any device) of attention's backward pass, the norm and the 8-bit product, with
bounds on the error that float arithmetic may make.

A bound is computed next to the value: every sum of n products in float is off by at most (n + 2) U times the sum
of the absolute products, U = 2^-24, and an error of the summands is carried through.  A type of fewer bits rounds
by half a step, eps / 2 of the value (bf16: 2^-8).
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def ball_rows(perm, npad, m):
    """[balls, m] rows (int64, -1 dummies) of a slot map, or of the identity."""
    if perm is None:
        return torch.arange(npad).view(-1, m)
    return perm[:npad].long().cpu().view(-1, m)


def attention_backward(Q, K, V, dO, balls, operand_half=0.0, out_half=U):
    """(dQ, dK, dV) and their bounds, float64, zero in rows no ball names.  operand_half: relative rounding of P and
    dS as operands of the last products."""
    Q, K, V, dO = (t.detach().double().cpu() for t in (Q, K, V, dO))
    d = Q.shape[2]
    sc = 1 / math.sqrt(d)
    grads = [torch.zeros_like(Q) for _ in range(3)]
    bounds = [torch.zeros_like(Q) for _ in range(3)]
    for idx in balls:
        idx = idx[idx >= 0]
        n = len(idx)
        if n == 0:
            continue
        q, k, v, g = (t[idx].transpose(0, 1) for t in (Q, K, V, dO))  # [H, n, d]
        s = q @ k.transpose(1, 2) * sc
        p = torch.softmax(s, 2)
        dp = g @ v.transpose(1, 2)
        delta = (p * dp).sum(2, keepdim=True)
        ds = p * (dp - delta)
        dv, dq, dk = p.transpose(1, 2) @ g, ds @ k * sc, ds.transpose(1, 2) @ q * sc
        # bounds: logits, probabilities (relative), dP, delta, dS
        es = (d + 4) * U * (q.abs() @ k.abs().transpose(1, 2)) * sc + 4 * U * s.abs()
        ep = 2 * es.amax(2, keepdim=True) + (n + 16) * U
        eg = (d + 2) * U * (g.abs() @ v.abs().transpose(1, 2))
        ed = (p * (ep * dp.abs() + eg)).sum(2, keepdim=True) + (n + 4) * U * (p * dp.abs()).sum(2, keepdim=True)
        eds = p * (ep * (dp - delta).abs() + eg + ed + 4 * U * (dp.abs() + delta.abs())) + operand_half * ds.abs()
        epp = (ep + operand_half) * p
        bv = epp.transpose(1, 2) @ g.abs() + (n + 2) * U * (p.transpose(1, 2) @ g.abs())
        bq = sc * (eds @ k.abs() + (n + 4) * U * (ds.abs() @ k.abs()))
        bk = sc * (eds.transpose(1, 2) @ q.abs() + (n + 4) * U * (ds.abs().transpose(1, 2) @ q.abs()))
        for o, b, t, e in zip(grads, bounds, (dq, dk, dv), (bq, bk, bv)):
            o[idx] = t.transpose(0, 1)
            # the result's rounding, and that of what is below the smallest normal numbers
            b[idx] = (1.01 * e + out_half * 1.01 * t.abs() + 1e-37).transpose(0, 1)
    return grads, bounds


def rms_norm(h, w, eps):
    """Norm of the stored stream h, with the bound of its float computation (before rounding to a type)."""
    h = h.detach().double().cpu()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double().cpu()
    return y, (h.shape[1] + 16) * U * y.abs()


def rms_norm_backward(dY, h, w, dH, eps):
    """(dX, dw) and the bounds of their float computation."""
    dY, h = dY.detach().double().cpu(), h.detach().double().cpu()
    rows, C = h.shape
    rs = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    g = dY if w is None else dY * w.double().cpu()
    dx = rs * (g - h * rs * rs * (g * h).mean(1, keepdim=True))
    bx = (2 * C + 32) * U * rs * (g.abs() + h.abs() * rs * rs * (g * h).abs().mean(1, keepdim=True))
    if dH is not None:
        dx = dx + dH.double().cpu()
        bx = bx + 2 * U * dx.abs()
    terms = dY * h * rs
    return dx, (terms).sum(0), bx, (rows + C + 32) * U * terms.abs().sum(0)


def project_i8(Xq, xs, Wq, ws):
    return (Xq.double().cpu() @ Wq.double().cpu().T) * xs.double().cpu()[:, None] * ws.double().cpu()[None, :]


def within(got, want, bound):
    """Every element of got within bound of want (both float64, CPU)."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), f"{int((~torch.isfinite(got)).sum())} values are not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (f"{int((over > 0).sum())} of {got.numel()} elements off, worst "
                               f"{float((got - want).abs().max()):.3e} (bound there "
                               f"{float(bound.flatten()[over.argmax()] if bound.numel() > 1 else bound):.3e})")
