"""The 8-bit Q/K/V projection and the pre-norm layer built on it, on the GPU against float64.

The product of 8-bit integers is exact, so a result is off by the three roundings of float (the sum as a float, two
scales: 3 x 2^-24) and by half a step of its type.
"""
import numpy as np
import pytest
import torch

import plain64
import workloads
from plain64 import HALF, U

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _ints(rows, C, seed, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-128 if full else -127, 128, (rows, C), generator=g, device="cuda").to(torch.int8)
    s = torch.exp(torch.randn(rows, generator=g, device="cuda"))
    return q, s


def _perm(rows, npad, seed):
    g = np.random.Generator(np.random.PCG64(seed))
    p = np.full(npad, -1, np.int32)
    p[np.sort(g.permutation(npad)[:rows])] = g.permutation(rows)
    return torch.from_numpy(p).cuda()


def _check(x, w, H, d, dtype, perm=None, inv=None):
    rows = x[0].shape[0]
    npad = rows if perm is None else perm.numel()
    out = tuple(torch.full((npad, H, d), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    bts.bt_qkv_project_i8(*x, *w, H, d, dtype=dtype, perm=perm, inv=inv, out=out)
    assert bts.bt_last_device_status() == 0
    want = plain64.project_i8(*x, *w)
    for t, got in enumerate(out):
        y = want[:, t * H * d:(t + 1) * H * d].reshape(rows, H, d)
        if perm is not None:
            p = perm.long().cpu()
            y = torch.where((p >= 0)[:, None, None], y[p.clamp(min=0)], 0.0)
        plain64.within(got, y, 1.01 * (3 * U + (HALF[dtype] if dtype == BF16 else 0)) * y.abs() + 1e-38)
    return out


# every width of load, rows from one up, K tails, columns that end inside a chunk
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C,H,d", [(1, 256, 8, 32), (1, 1, 1, 1), (3, 5, 2, 3), (7, 512, 8, 64), (8, 100, 3, 64),
                                        (9, 48, 1, 32), (32, 17, 2, 32), (33, 64, 2, 32), (40, 130, 5, 24),
                                        (127, 256, 4, 32), (128, 128, 2, 32), (300, 16, 1, 8), (1000, 272, 8, 32),
                                        (777, 1040, 3, 64), (260, 2064, 5, 64), (500, 36, 4, 32), (2500, 256, 8, 32),
                                        (600, 512, 8, 64), (520, 640, 16, 32), (129, 15, 3, 20)])
def test_against_float64(rows, C, H, d, dtype):
    x, w = _ints(rows, C, rows + C), _ints(3 * H * d, C, H + d)
    _check(x, w, H, d, dtype)
    npad = max(16, rows + rows // 3)
    perm = _perm(rows, npad, rows)
    _check(x, w, H, d, dtype, perm=perm)
    _check(x, w, H, d, dtype, perm=perm, inv=bts.bt_invert_perm(perm, rows))


def test_largest_sums():
    # all values at their ends, -128 among them: the largest sums are exact
    for rows, C in ((4, 65536), (200, 65536)):
        x, w = _ints(rows, C, 1, full=True), _ints(24, C, 2, full=True)
        x[0][0] = -128
        w[0][0] = -128
        x[0][1] = 127
        _check(x, w, 1, 8, F32)


def test_many_rows():
    x, w = _ints(70001, 128, 3), _ints(3 * 2 * 32, 128, 4)
    _check(x, w, 2, 32, BF16, perm=_perm(70001, 80000, 5))


def test_no_rows():
    w = _ints(96, 64, 1)
    x = (torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert bts.bt_qkv_project_i8(*x, *w, 1, 32)[0].shape == (0, 1, 32)
    out = tuple(torch.full((256, 1, 32), 7.0, dtype=BF16, device="cuda") for _ in range(3))
    perm = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    bts.bt_qkv_project_i8(*x, *w, 1, 32, perm=perm, inv=torch.empty(0, dtype=torch.int32, device="cuda"), out=out)
    assert all((t == 0).all() for t in out)  # dummy slots


@pytest.mark.parametrize("off", [1, 4, 16])
def test_any_alignment(off):
    rows, C, H, d = 200, 64, 2, 32
    xb, wb = _ints(1, rows * C + 16, 6)[0].flatten(), _ints(1, 192 * C + 16, 7)[0].flatten()
    x = (xb[off:off + rows * C].view(rows, C), _ints(rows, 1, 8)[1])
    w = (wb[off:off + 192 * C].view(192, C), _ints(192, 1, 9)[1])
    for dtype in (F32, BF16):
        _check(x, w, H, d, dtype)
        buf = torch.zeros(3, rows * H * d + 8, dtype=dtype, device="cuda")
        got = tuple(b[1:1 + rows * H * d].view(rows, H, d) for b in buf)  # outputs at odd addresses
        bts.bt_qkv_project_i8(*x, *w, H, d, dtype=dtype, out=got)
        for a, b in zip(got, bts.bt_qkv_project_i8(*x, *w, H, d, dtype=dtype)):
            assert torch.equal(a, b)
        assert (buf[:, 0] == 0).all() and (buf[:, 1 + rows * H * d:] == 0).all()


def test_scales_not_finite_stay_in_their_row_and_channel():
    for rows in (9, 400):
        x, w = _ints(rows, 128, 10), _ints(192, 128, 11)
        clean = bts.bt_qkv_project_i8(*x, *w, 2, 32)
        x[1][5] = float("nan")
        x[0][5] = 0
        got = bts.bt_qkv_project_i8(*x, *w, 2, 32)
        keep = torch.arange(rows, device="cuda") != 5
        for a, b in zip(got, clean):
            assert torch.isnan(a[5]).all() and torch.equal(a[keep], b[keep])


def test_bad_slot_is_recorded_not_written():
    for rows in (20, 1000):
        x, w = _ints(rows, 128, 12), _ints(192, 128, 13)
        perm = _perm(rows, rows, 14)
        inv = bts.bt_invert_perm(perm, rows)
        lost = int(inv[7])
        for bad in (rows, -1, 2 ** 31 - 1):
            inv[7] = bad
            out = tuple(torch.full((rows, 2, 32), 7.0, dtype=BF16, device="cuda") for _ in range(3))
            got = bts.bt_qkv_project_i8(*x, *w, 2, 32, perm=perm, inv=inv, out=out)
            assert bts.bt_last_device_status() == 8 and bts.bt_last_device_status() == 0
            want = bts.bt_qkv_project_i8(*x, *w, 2, 32, perm=perm)
            keep = torch.arange(rows, device="cuda") != lost
            for a, b in zip(got, want):
                assert (a[lost] == 7.0).all() and torch.equal(a[keep], b[keep])


def test_streams_and_capture():
    x, w = _ints(5000, 256, 15), _ints(768, 256, 16)
    perm = _perm(5000, 6000, 17)
    want = bts.bt_qkv_project_i8(*x, *w, 8, 32, perm=perm)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    got = [bts.bt_qkv_project_i8(*x, *w, 8, 32, perm=perm, stream=s) for s in ss for _ in range(2)]
    torch.cuda.synchronize()
    inv = bts.bt_invert_perm(perm, 5000)
    out = tuple(torch.empty_like(t) for t in want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bts.bt_qkv_project_i8(*x, *w, 8, 32, perm=perm, inv=inv, out=out)
    g.replay()
    torch.cuda.synchronize()
    for o in got + [out]:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def _layer_inputs(rows, C, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn(rows, C, generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    wt = torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5
    return x, r, gamma, wt


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C,H,d,m", [(3000, 256, 8, 32, 128), (700, 64, 4, 32, 16), (500, 96, 3, 64, 64),
                                          (20, 128, 2, 32, 16), (1, 64, 2, 32, 16), (300, 50, 2, 32, 256)])
def test_layer_equals_its_steps(rows, C, H, d, m, dtype):
    x, r, gamma, wt = _layer_inputs(rows, C, H, d, dtype, rows)
    pts = torch.from_numpy(workloads.uniform_cloud(rows, C)).cuda()
    perm, _ = bts.bt_build_segmented(pts, [0, rows], m)
    wq, ws = bts.bt_quantize_i8(wt)
    for res in (r, None):
        O, h = bts.bt_projected_ball_attention_i8(x, perm, wq, ws, m, H, d, weight=gamma, residual=res)
        assert bts.bt_last_device_status() == 0
        xq, xs, h2 = bts.bt_rms_norm_i8(x, gamma, residual=res)
        q, k, v = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype)
        assert torch.equal(h, h2)
        assert torch.equal(O, bts.bt_ball_attention(q, k, v, perm, m))
    O, _ = bts.bt_projected_ball_attention_i8(x, None, wq, ws, 1, H, d, weight=gamma)  # balls of one row: V itself
    xq, xs, _ = bts.bt_rms_norm_i8(x, gamma)
    v = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype)[2]
    assert ((O.double() - v.double()).abs() <= 2 * HALF[dtype] * v.double().abs()).all()


def test_layer_near_the_layer_in_16_bits():
    # 8 bits cost half a step of 1/127 of the row's maximum (about 3 to 4 standard deviations) on each operand:
    # 4 / 127 / sqrt(12) = 0.9 % of a value's deviation each, 1.3 % of Q, K and V together; logits of deviation 1
    # move by that (twice, for q and k), and so does O relative to its own size: 5 % bounds the sum in norm
    rows, C, H, d, m = 4096, 256, 8, 32, 128
    x, r, gamma, wt = _layer_inputs(rows, C, H, d, BF16, 3)
    pts = torch.from_numpy(workloads.uniform_cloud(rows, 3)).cuda()
    perm = bts.bt_build(pts, m)
    wq, ws = bts.bt_quantize_i8(wt)
    O, h = bts.bt_projected_ball_attention_i8(x, perm, wq, ws, m, H, d, weight=gamma, residual=r)
    y, h2 = bts.bt_rms_norm(x, gamma, residual=r)
    ref = bts.bt_projected_ball_attention(y, perm, wt.to(BF16), m, H, d)
    assert torch.equal(h, h2)
    assert (O.double() - ref.double()).norm() <= 0.05 * ref.double().norm()


def test_a_training_step_of_the_layer_against_differentiation():
    # norm -> projection -> ball attention forward, and its backward pass through the library's gradients, in float:
    # against differentiation of the same chain in float64
    rows, C, H, d, m, eps = 512, 64, 2, 32, 32, 1e-6
    x, r, gamma, wt = _layer_inputs(rows, C, H, d, F32, 4)
    pts = torch.from_numpy(workloads.uniform_cloud(rows, 5)).cuda()
    perm = bts.bt_build(pts, m)
    g = torch.Generator(device="cuda").manual_seed(6)
    dO = torch.randn(rows, H, d, generator=g, device="cuda")
    dH = torch.randn(rows, C, generator=g, device="cuda")
    y, h = bts.bt_rms_norm(x, gamma, residual=r, eps=eps)
    qkv = (y @ wt.T).view(rows, 3, H, d).unbind(1)
    grads = bts.bt_ball_attention_backward(*(t.contiguous() for t in qkv), dO, perm, m)
    dqkv = torch.stack(grads, 1).view(rows, 3 * H * d)
    dW, dY = dqkv.T @ y, dqkv @ wt
    dX, dgamma = bts.bt_rms_norm_backward(dY, h, gamma, dH=dH, eps=eps)

    leaves = [t.double().requires_grad_(True) for t in (x, r, gamma, wt)]
    hh = leaves[0] + leaves[1]
    yy = hh / torch.sqrt(hh.square().mean(1, keepdim=True) + eps) * leaves[2]
    q, k, v = (t[perm.long()].view(-1, m, H, d).transpose(1, 2) for t in (yy @ leaves[3].T).view(rows, 3, H, d).unbind(1))
    o = torch.softmax(q @ k.transpose(2, 3) / d ** 0.5, 3) @ v
    loss = (o * dO.double()[perm.long()].view(-1, m, H, d).transpose(1, 2)).sum() + (hh * dH.double()).sum()
    want = torch.autograd.grad(loss, leaves)
    # a chain of five float sums of at most 512 terms, each within (n + 2) 2^-24 of its absolute products; their
    # ratio to the results' norm is of order sqrt(n): 1e-4 bounds the chain in norm
    for got, w in zip((dX, dX, dgamma, dW), want):
        assert (got.double() - w).norm() <= 1e-4 * w.norm()


def test_refusals():
    x, w = _ints(64, 64, 20), _ints(192, 64, 21)
    call = bts.bt_qkv_project_i8
    with pytest.raises(TypeError):
        call(x[0].float(), x[1], *w, 2, 32)
    with pytest.raises(TypeError):
        call(*x, w[0], w[1].double(), 2, 32)
    with pytest.raises(TypeError):
        call(*x, *w, 2, 32, dtype=torch.float16)
    with pytest.raises(ValueError):
        call(*x, *w, 2, 16)
    with pytest.raises(ValueError):
        call(x[0], x[1][:10], *w, 2, 32)
    with pytest.raises(ValueError):
        call(x[0].cpu(), x[1], *w, 2, 32)
    out = torch.empty(64, 2, 32, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        call(*x, *w, 2, 32, out=(out, out, out))
    perm = _perm(64, 64, 1)
    with pytest.raises(TypeError):
        call(*x, *w, 2, 32, perm=perm, inv=perm.long())
    xf, gamma = torch.zeros(64, 64, device="cuda", dtype=BF16), torch.ones(64, device="cuda")
    with pytest.raises(bts.BtsError) as e:
        bts.bt_projected_ball_attention_i8(xf, perm, *w, 32, 2, 32, weight=gamma,
                                           work=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == "BT_ERR_WORKSPACE"
    with pytest.raises(bts.BtsError) as e:
        bts.bt_projected_ball_attention_i8(xf, perm, *w, 48, 2, 32, weight=gamma)
    assert e.value.status == "BT_ERR_SHAPE"


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_rows(dtype):
    # an empty batch: every call returns results of no rows, the gradient of the weight is zero
    x, r = (torch.empty((0, 64), dtype=dtype, device="cuda") for _ in range(2))
    w8, ws = bts.bt_quantize_i8(torch.ones((192, 64), dtype=dtype, device="cuda"))
    weight = torch.ones(64, device="cuda")
    y, h = bts.bt_rms_norm(x, weight, r)
    xq, xs, _ = bts.bt_rms_norm_i8(x, weight, r)
    dx, dw = bts.bt_rms_norm_backward(y, h, weight)
    assert y.shape == h.shape == xq.shape == dx.shape == (0, 64) and xs.shape == (0,) and (dw == 0).all()
    for perm in (None, torch.empty(0, dtype=torch.int32, device="cuda")):
        q, k, v = bts.bt_qkv_project_i8(xq, xs, w8, ws, 2, 32, dtype, perm)
        assert q.shape == k.shape == v.shape == (0, 2, 32)
        assert all(g.shape == q.shape for g in bts.bt_ball_attention_backward(q, k, v, q, perm, 16))
        o, h = bts.bt_projected_ball_attention_i8(x, perm, w8, ws, 16, 2, 32, weight, r)
        assert o.shape == (0, 2, 32) and h.shape == (0, 64)
    torch.cuda.synchronize()
    assert bts.bt_last_device_status() == 0
