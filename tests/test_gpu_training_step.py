"""The autograd functions that the README shows, in a training step of a layer: norm with the residual, projection, ball
attention, and a loss on the output and on the residual stream, against differentiation of the chain in float64.

Float: five sums of at most 768 terms, each within (n + 2) 2^-24 of its absolute products; their ratio to the results'
norm is of order sqrt(n): 1e-4 bounds the chain in norm.
bf16: a rounding is off by at most 2^-8 of a value, evenly, so by e = 2^-8 / sqrt(3) in norm, and errors add at most
linearly.  h and Y: 2 e.  Q, K and V: 3 e.  Scores, of a deviation of about 1, from Q and K: 6 e.  P, from the scores and
their sum: 12 e; as an operand 13 e, and dV with its own rounding 14 e.  dP: 3 e, twice in dP - delta; dS: 12 + 6 + 1 = 19 e.
dQ and dK, with K or Q and their rounding: 23 e.  The gradients of the weights, with Y: 26 e; dY, rounded: 24 e; dX and
the gradient of the norm's weight, with h: 27 e = 0.061.
"""
import os
import re

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def shown():
    text = open(os.path.join(ROOT, "README.md")).read()
    code, = re.findall(r"```python\n(.*?)```", text, re.S)
    names = {}
    exec(compile(code, "README.md", "exec"), names)
    return names


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C,H,d,m", [(1024, 256, 8, 32, 128), (512, 64, 2, 32, 32), (768, 96, 3, 64, 64),
                                          (1024, 128, 2, 64, 256)])
def test_gradients_of_a_layer(shown, rows, C, H, d, m, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + m)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    x, r = (normal(rows, C).to(dtype).requires_grad_(True) for _ in range(2))
    gamma = (1 + 0.2 * normal(C)).requires_grad_(True)
    wt = (normal(3 * H * d, C) / C ** 0.5).to(dtype).requires_grad_(True)
    dO, dH = normal(rows, H, d).to(dtype), normal(rows, C).to(dtype)
    eps = 1e-6
    pts = torch.from_numpy(workloads.uniform_cloud(rows, 5)).cuda()
    perm, _ = bts.bt_build_segmented(pts, [0, rows], m)

    y, h = shown["Norm"].apply(x, r, gamma, eps)
    q, k, v = torch.nn.functional.linear(y, wt).view(rows, 3, H, d).unbind(1)
    o = shown["BallAttention"].apply(q, k, v, perm, m)
    got = torch.autograd.grad((o.float() * dO.float()).sum() + (h.float() * dH.float()).sum(), (x, r, gamma, wt))
    assert bts.bt_last_device_status() == 0
    for a, b in zip(got, (x, r, gamma, wt)):
        assert a.dtype == b.dtype and a.shape == b.shape

    leaves = [t.detach().double().requires_grad_(True) for t in (x, r, gamma, wt)]
    hh = leaves[0] + leaves[1]
    yy = hh / torch.sqrt(hh.square().mean(1, keepdim=True) + eps) * leaves[2]
    real = perm >= 0
    q, k, v = (t[perm.clamp(min=0).long()].view(-1, m, H, d).transpose(1, 2)
               for t in (yy @ leaves[3].T).view(rows, 3, H, d).unbind(1))
    s = (q @ k.transpose(2, 3) / d ** 0.5).masked_fill(~real.view(-1, 1, 1, m), -1e300)
    oo = (torch.softmax(s, 3) @ v).transpose(1, 2).reshape(-1, H, d)[real]
    want = torch.autograd.grad((oo * dO.double()[perm[real].long()]).sum() + (hh * dH.double()).sum(), leaves)
    tol = 1e-4 if dtype == F32 else 27 * 2.0 ** -8 / 3 ** 0.5
    for a, b in zip(got, want):
        err = float((a.double() - b).norm() / b.norm())
        print(f"relative error in norm {err:.2e}, bound {tol:.2e}")
        assert err <= tol
