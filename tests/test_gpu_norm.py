"""RMS norm with the residual's addition, its 8-bit output and its backward pass on the GPU against float64.

Bounds (plain64): a sum of C products in float is off by (C + 2) 2^-24 of the absolute products; results round by
half a step of their type.  8 bits: the scale is one division of a maximum, and a value is off by half a step of
the scale, and by the error of y itself.
"""
import pytest
import torch

import plain64
from plain64 import HALF, U

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (1, 256), (1, 8192), (2, 8), (3, 7), (5, 1000), (7, 1024), (33, 2050), (64, 129), (300, 64),
          (513, 250), (1000, 33), (4000, 128), (5000, 256), (1500, 4096), (70000, 16)]


def _rows(rows, C, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, C, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    return x.to(dtype)


def _weight(C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(C, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_norm(rows, C, dtype):
    x, r, w = _rows(rows, C, dtype, 1), _rows(rows, C, dtype, 2), _weight(C, 3)
    for res, wt, eps in ((r, w, 1e-6), (None, w, 1e-6), (r, None, 1e-2), (None, None, 1e-5)):
        y, h = bts.bt_rms_norm(x, wt, residual=res, eps=eps)
        want_h = x if res is None else (x.float() + res.float()).to(dtype)
        assert torch.equal(h, want_h)
        want, bound = plain64.rms_norm(want_h, wt, eps)
        plain64.within(y, want, 1.01 * bound + 1.01 * HALF[dtype] * want.abs() + 1e-38)


def _check_i8(q, s, y, bound):
    """8-bit rows and scales against float64 values y known to within `bound`."""
    assert (q >= -127).all()
    rel = (bound / y.abs().clamp(min=1e-300)).nan_to_num(0).amax(1)
    want = y.abs().amax(1) / 127
    plain64.within(s, want, (rel + 2 * U) * want + 1e-44)
    s = s.double().cpu()
    err = (q.double().cpu() * s[:, None] - y).abs()
    # half a step, the value's own error, and the quotient's rounding (at most 128 U of a step)
    assert (err <= (0.5 + 128 * U) * s[:, None] + bound + 1e-44).all(), float((err / s[:, None].clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_norm_and_quantisation_in_8_bits(rows, C, dtype):
    x, r, w = _rows(rows, C, dtype, 4), _rows(rows, C, dtype, 5), _weight(C, 6)
    for res, wt in ((r, w), (None, None)):
        q, s, h = bts.bt_rms_norm_i8(x, wt, residual=res)
        assert torch.equal(h, x if res is None else (x.float() + res.float()).to(dtype))
        _check_i8(q, s, *plain64.rms_norm(h, wt, 1e-6))
    q, s = bts.bt_quantize_i8(x)
    y = x.double().cpu()
    _check_i8(q, s, y, torch.zeros_like(y))
    # the scale and the values are single roundings: equal to torch's divisions (by a tensor: by a number, torch
    # multiplies with its reciprocal, which rounds twice)
    mx = x.float().abs().amax(1)
    want = mx / torch.full_like(mx, 127)
    assert torch.equal(s, want)
    assert torch.equal(q, torch.round(x.float() / torch.where(want > 0, want, 1)[:, None]).to(torch.int8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_backward(rows, C, dtype):
    h, dY, dH, w = _rows(rows, C, dtype, 7), _rows(rows, C, dtype, 8), _rows(rows, C, dtype, 9), _weight(C, 10)
    for wt, up in ((w, dH), (w, None), (None, dH)):
        dx, dw = bts.bt_rms_norm_backward(dY, h, wt, dH=up)
        wx, ww, bx, bw = plain64.rms_norm_backward(dY, h, wt, up, 1e-6)
        plain64.within(dx, wx, 1.01 * bx + 1.01 * HALF[dtype] * wx.abs() + 1e-38)
        if wt is None:
            assert dw is None
        else:
            plain64.within(dw, ww, 1.01 * bw + 1e-38)


def test_backward_by_differences_of_the_forward_pass():
    rows, C = 16, 48
    x, dY, w = _rows(rows, C, F32, 11), _rows(rows, C, F32, 12), _weight(C, 13)
    dx, dw = bts.bt_rms_norm_backward(dY, x, w, eps=1e-3)
    t = 2.0 ** -8
    for i in range(2):
        dirn = torch.randn_like(x) if i == 0 else torch.randn_like(w)
        f = []
        for s in (1, -1):
            y, _ = bts.bt_rms_norm(x + s * t * dirn if i == 0 else x, w if i == 0 else w + s * t * dirn, eps=1e-3)
            f.append(float((y.double() * dY.double()).sum()))
        want = float(((dx if i == 0 else dw).double() * dirn.double()).sum())
        mass = float((dY.double().abs() * y.double().abs()).sum())
        # float rounding of y over 2 t, and t^2 times the curvature of rows whose norm is of order 0.1 or more
        assert abs((f[0] - f[1]) / (2 * t) - want) <= mass * ((C + 16) * U / t + 100 * t * t)


def test_rows_of_zeros_and_of_values_not_finite():
    for dtype in (F32, BF16):
        x = _rows(6, 96, dtype, 14)
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 95] = float("inf")
        x[4, 0] = -float("inf")
        q, s = bts.bt_quantize_i8(x)
        assert s[1] == 0 and (q[1] == 0).all()
        for i in (2, 3, 4):
            assert torch.isnan(s[i]) and (q[i] == 0).all()
        assert torch.isfinite(s[[0, 5]]).all()
        q, s, _ = bts.bt_rms_norm_i8(x)
        assert s[1] == 0 and (q[1] == 0).all()
        assert all(torch.isnan(s[i]) and (q[i] == 0).all() for i in (2, 3, 4))
        y, _ = bts.bt_rms_norm(x)
        assert (y[1] == 0).all() and torch.isfinite(y[[0, 5]]).all()
        assert all(not torch.isfinite(y[i]).all() for i in (2, 3, 4))


def test_extreme_scales():
    # rows of the smallest and largest magnitudes whose squares float holds; and for the quantisation, any
    for dtype in (F32, BF16):
        x = _rows(4, 64, dtype, 15).float()
        for v in (1e-15, 1e15):
            y, _ = bts.bt_rms_norm((x * v).to(dtype), eps=0.0)
            want, bound = plain64.rms_norm((x * v).to(dtype), None, 0.0)
            plain64.within(y, want, 1.01 * bound + 1.01 * HALF[dtype] * want.abs())
        for v in (1e-35, 1e36):
            z = (x * v).to(dtype)
            q, s = bts.bt_quantize_i8(z)
            _check_i8(q, s, z.double().cpu(), torch.zeros(4, 64, dtype=torch.float64))


def test_no_rows():
    for dtype in (F32, BF16):
        x = torch.empty(0, 64, dtype=dtype, device="cuda")
        w = _weight(64, 1)
        assert bts.bt_rms_norm(x, w, residual=x)[0].shape == (0, 64)
        assert bts.bt_rms_norm_i8(x, w)[1].shape == (0,)
        assert bts.bt_quantize_i8(x)[0].shape == (0, 64)
        dx, dw = bts.bt_rms_norm_backward(x, x, w, dw=torch.full((64,), 7.0, device="cuda"))
        assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_any_alignment_and_in_place(dtype):
    rows, C = 70, 96
    base = [_rows(1, rows * C + 8, dtype, 20 + i).flatten() for i in range(3)]
    for off in (0, 1, 2, 3):
        x, r, dy = (b[off:off + rows * C].view(rows, C) for b in base)
        w = _weight(C + 4, 2)[off:off + C]
        y, h = bts.bt_rms_norm(x, w, residual=r)
        q, s, _ = bts.bt_rms_norm_i8(x, w, residual=r)
        dx, dw = bts.bt_rms_norm_backward(dy, x, w, dH=r)
        want, bound = plain64.rms_norm(h, w, 1e-6)
        plain64.within(y, want, 1.01 * bound + 1.01 * HALF[dtype] * want.abs())
        _check_i8(q, s, want, bound)
        # into the residual and the input; dX into dH and into dY
        x2, r2 = x.clone(), r.clone()
        bts.bt_rms_norm(x2, w, residual=r2, out=x2, hout=r2)
        x3, r3 = x.clone(), r.clone()
        bts.bt_rms_norm(x3, w, residual=r3, out=r3, hout=x3)
        wx, ww, bx, bw = plain64.rms_norm_backward(dy, x, w, r, 1e-6)
        plain64.within(dx, wx, 1.01 * bx + 1.01 * HALF[dtype] * wx.abs())
        plain64.within(dw, ww, 1.01 * bw)
        if off == 0:  # the same split of the row: equal bits
            assert torch.equal(x2, y) and torch.equal(r2, h) and torch.equal(r3, y) and torch.equal(x3, h)
            for into in (r.clone(), dy.clone()):
                a, b = (dy, into) if into.equal(r) else (into, r)
                assert torch.equal(bts.bt_rms_norm_backward(a, x, w, dH=b, out=into)[0], dx)


def test_equal_calls_streams_and_capture():
    x, dY, w = _rows(3000, 256, BF16, 30), _rows(3000, 256, BF16, 31), _weight(256, 32)
    want = bts.bt_rms_norm_backward(dY, x, w)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    got = [bts.bt_rms_norm_backward(dY, x, w, stream=s) for s in ss for _ in range(2)]
    torch.cuda.synchronize()
    for o in got:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, out, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(256, device="cuda")
    ws = torch.empty(bts.bt_rms_norm_backward_workspace_size(3000, 256), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bts.bt_rms_norm(x, w, out=y)
        bts.bt_rms_norm_backward(dY, x, w, out=out, dw=dw, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(dw, want[1])
    assert torch.equal(y, bts.bt_rms_norm(x, w)[0])


def test_refusals():
    x, w = _rows(8, 64, BF16, 40), _weight(64, 41)
    with pytest.raises(TypeError):
        bts.bt_rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        bts.bt_rms_norm(x, w.to(BF16))
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x, w, residual=x[:4])
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x, w, hout=torch.empty_like(x))
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x[:, ::2], w[:32].contiguous())
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x.cpu(), w)
    out = torch.empty_like(x)
    with pytest.raises(ValueError):
        bts.bt_rms_norm(x, w, residual=x, out=out, hout=out)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(bts.BtsError) as e:
            bts.bt_rms_norm(x, w, eps=eps)
        assert e.value.status == "BT_ERR_ARG"
    wide = torch.zeros(1, 8193, dtype=BF16, device="cuda")
    for call in (bts.bt_rms_norm, bts.bt_rms_norm_i8, bts.bt_quantize_i8):
        with pytest.raises(bts.BtsError) as e:
            call(wide)
        assert e.value.status == "BT_ERR_UNSUPPORTED"
    with pytest.raises(bts.BtsError) as e:
        bts.bt_rms_norm_backward(x, x, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == "BT_ERR_WORKSPACE"
    with pytest.raises(ValueError):
        bts.bt_rms_norm_backward(x, x, w, out=x)
