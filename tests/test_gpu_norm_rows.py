"""Rows whose length is no multiple of a vector: they begin and end inside one, next to other rows.

The same bounds as in test_gpu_norm; here for lengths from one element up, tensors that end inside a vector, results
that must leave what lies around them alone, and in-place calls, where a row's neighbours are written while it is read.
"""
import pytest
import torch

import plain64
from plain64 import HALF, U

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32
LENGTHS = [1, 2, 3, 5, 6, 7, 9, 15, 17, 31, 33, 63, 129, 257, 1001, 2047, 4097, 8191]


def _random(rows, C, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, C, generator=g, device="cuda").to(dtype)


def _inside(rows, C, dtype, fill):
    """An array between two guards (16 bytes aligned), and the whole."""
    whole = torch.full((32 + rows * C + 32,), fill, dtype=dtype, device="cuda")
    return whole[32:32 + rows * C].view(rows, C), whole


def _guards(whole, n, fill):
    assert (whole[:32] == fill).all() and (whole[32 + n:] == fill).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", LENGTHS)
def test_guards_and_values(C, dtype):
    for rows in (1, 2, 3, 8, 9, 41):
        n = rows * C
        x, _ = _inside(rows, C, dtype, float("nan"))  # what lies around the inputs must not count
        r, _ = _inside(rows, C, dtype, float("nan"))
        dy, _ = _inside(rows, C, dtype, float("nan"))
        for i, t in enumerate((x, r, dy)):
            t.copy_(_random(rows, C, dtype, C + i))
        w = 1 + 0.3 * torch.randn(C, generator=torch.Generator(device="cuda").manual_seed(C), device="cuda")
        y, yw = _inside(rows, C, dtype, 7.0)
        h, hw = _inside(rows, C, dtype, 7.0)
        bts.bt_rms_norm(x, w, residual=r, out=y, hout=h)
        assert torch.equal(h, (x.float() + r.float()).to(dtype))
        want, bound = plain64.rms_norm(h, w, 1e-6)
        plain64.within(y, want, 1.01 * bound + 1.01 * HALF[dtype] * want.abs() + 1e-38)
        _guards(yw, n, 7.0)
        _guards(hw, n, 7.0)
        q, qw = _inside(rows, C, torch.int8, 7)
        _, s, _ = bts.bt_rms_norm_i8(x, w, residual=r, out=q, hout=h)
        sd = s.double().cpu()
        err = (q.double().cpu() * sd[:, None] - want).abs()
        assert (err <= (0.5 + 128 * U) * sd[:, None] + bound + 1e-44).all()
        _guards(qw, n, 7)
        _guards(hw, n, 7.0)
        dx, dxw = _inside(rows, C, dtype, 7.0)
        _, dw = bts.bt_rms_norm_backward(dy, h, w, dH=r, out=dx)
        wx, ww, bx, bw = plain64.rms_norm_backward(dy, h, w, r, 1e-6)
        plain64.within(dx, wx, 1.01 * bx + 1.01 * HALF[dtype] * wx.abs() + 1e-38)
        plain64.within(dw, ww, 1.01 * bw + 1e-38)
        _guards(dxw, n, 7.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", [(5000, 3), (3000, 13), (2000, 33), (700, 257), (300, 1001)])
def test_in_place(rows, C, dtype):
    x, r, w = _random(rows, C, dtype, 1), _random(rows, C, dtype, 2), torch.ones(C, device="cuda")
    y, h = bts.bt_rms_norm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    bts.bt_rms_norm(x2, w, residual=r2, out=x2, hout=r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    q, s, _ = bts.bt_rms_norm_i8(x, w, residual=r)
    x3 = x.clone()
    q2, s2, _ = bts.bt_rms_norm_i8(x3, w, residual=r, hout=x3)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(x3, h)
    dx, dw = bts.bt_rms_norm_backward(y, h, w, dH=r)
    for into in (y.clone(), r.clone()):
        a, b = (into, r) if into.equal(y) else (y, into)
        dx2, dw2 = bts.bt_rms_norm_backward(a, h, w, dH=b, out=into)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_rows_than_groups(dtype):
    # a group walks many rows, whose shift is the same; columns of dw from groups of every shift
    for rows, C in ((200000, 7), (60000, 45), (20000, 333), (9000, 1029)):
        h, dy = _random(rows, C, dtype, C), _random(rows, C, dtype, C + 1)
        w = 1 + 0.1 * torch.arange(C, device="cuda") / C
        dx, dw = bts.bt_rms_norm_backward(dy, h, w)
        wx, ww, bx, bw = plain64.rms_norm_backward(dy, h, w, None, 1e-6)
        plain64.within(dx, wx, 1.01 * bx + 1.01 * HALF[dtype] * wx.abs() + 1e-38)
        plain64.within(dw, ww, 1.01 * bw + 1e-38)


def test_refusals_of_shared_memory():
    x, w = _random(8, 64, BF16, 1), torch.ones(64, device="cuda")
    flat = torch.zeros(8 * 64 + 64, dtype=BF16, device="cuda")
    a, b = flat[:512].view(8, 64), flat[64:576].view(8, 64)
    for call in (lambda: bts.bt_rms_norm(a, w, out=b), lambda: bts.bt_rms_norm(x, w, residual=a, hout=b),
                 lambda: bts.bt_rms_norm(x, w, residual=x, out=a, hout=a),
                 lambda: bts.bt_rms_norm_backward(x, a, w, out=a), lambda: bts.bt_rms_norm_backward(a, x, w, out=b)):
        with pytest.raises(ValueError):
            call()
