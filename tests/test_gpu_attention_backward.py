"""Backward pass of ball attention on the GPU against the float64 formula, element by element.

The bounds are derived in plain64.attention_backward: float arithmetic throughout, and for the tensor-core shapes
(bf16, m <= 128) one rounding of P and of dS to bf16 (2^-8 of each) before the last three products; the results
round to their type.
"""
import numpy as np
import pytest
import torch

import plain64
import workloads

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(rows, H, d, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(rows, H, d, generator=g, device="cuda") * scale).to(dtype) for _ in range(4)]


def _perm(rows, npad, seed, dummies="end"):
    g = np.random.Generator(np.random.PCG64(seed))
    p = np.full(npad, -1, np.int32)
    at = np.arange(rows) if dummies == "end" else np.sort(g.permutation(npad)[:rows])
    p[at] = g.permutation(rows)
    return torch.from_numpy(p).cuda()


def _check(x, perm, m, npad=None):
    Q, K, V, dO = x
    out = tuple(torch.full_like(Q, 7.0) for _ in range(3))
    got = bts.bt_ball_attention_backward(Q, K, V, dO, perm, m, out=out, npad=npad)
    assert bts.bt_last_device_status() == 0
    n = npad if npad is not None else (Q.shape[0] if perm is None else perm.numel())
    balls = plain64.ball_rows(perm, n, m)
    half = plain64.HALF[BF16] if Q.dtype == BF16 else 0.0
    want, bound = plain64.attention_backward(Q, K, V, dO, balls, operand_half=half,
                                             out_half=plain64.HALF[Q.dtype])
    named = torch.zeros(Q.shape[0], dtype=torch.bool)
    named[balls[balls >= 0]] = True
    for a, b, e in zip(got, want, bound):
        assert (a[~named] == 7.0).all()  # rows no slot names
        plain64.within(a[named], b[named], e[named])
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,d,H", [(32, 32, 2), (128, 32, 8), (128, 64, 3), (64, 32, 3), (16, 64, 1), (1, 32, 2),
                                   (2, 64, 2), (7, 32, 1), (33, 32, 2), (48, 64, 5), (100, 32, 4), (127, 64, 2),
                                   (129, 32, 2), (200, 64, 1), (256, 32, 3), (256, 64, 2)])
def test_against_float64(m, d, H, dtype):
    balls = max(3, 300 // m)
    rows = balls * m
    _check(_inputs(rows, H, d, dtype, m * d + H), _perm(rows, rows, m), m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,npad,m,dummies", [(1, 128, 128, "end"), (130, 512, 128, "end"), (5, 64, 16, "end"),
                                                 (77, 256, 32, "any"), (200, 384, 128, "any"), (3, 400, 100, "any"),
                                                 (90, 512, 256, "any"), (1, 1, 1, "end"), (37, 60, 20, "any")])
def test_dummies(rows, npad, m, dummies, dtype):
    _check(_inputs(rows, 2, 32, dtype, rows), _perm(rows, npad, npad, dummies), m)
    _check(_inputs(rows, 3, 64, dtype, rows + 1), _perm(rows, npad, npad + 1, dummies), m)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_identity_order_and_rows_no_slot_names(dtype):
    x = _inputs(300, 2, 32, dtype, 3)
    _check(x, None, 32, npad=288)
    _check(x, torch.arange(256, dtype=torch.int32, device="cuda"), 64)
    _check(x, _perm(300, 320, 4), 32, npad=160)  # a part of the slots


def test_all_dummies_writes_nothing():
    for dtype in (F32, BF16):
        _check(_inputs(10, 2, 32, dtype, 5), torch.full((256,), -1, dtype=torch.int32, device="cuda"), 64)


def test_no_slots_or_rows():
    x = [torch.empty(0, 2, 32, device="cuda", dtype=BF16)] * 4
    out = bts.bt_ball_attention_backward(*x, None, 16)
    assert all(t.shape == (0, 2, 32) for t in out)
    y = _inputs(4, 2, 32, BF16, 1)
    out = tuple(torch.full_like(y[0], 7.0) for _ in range(3))
    bts.bt_ball_attention_backward(*y, torch.empty(0, dtype=torch.int32, device="cuda"), 16, out=out)
    assert all((t == 7.0).all() for t in out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-3, 6.0])
def test_flat_and_peaked_softmax(dtype, scale):
    # nearly equal weights, and logits of a few hundred: one key takes almost everything
    _check(_inputs(256, 2, 32, dtype, 9, scale), _perm(256, 256, 9), 128)
    _check(_inputs(256, 2, 64, dtype, 10, scale), _perm(256, 256, 10), 32)


def test_equal_keys():
    # all keys equal: P is 1/n and dS sums to nothing along a row
    for dtype in (F32, BF16):
        x = _inputs(128, 2, 32, dtype, 11)
        x[1][:] = x[1][:1]
        _check(x, _perm(128, 128, 2), 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,d", [(16, 32), (32, 64), (50, 32), (64, 64), (128, 32)])
def test_values_not_finite_stay_in_their_ball_and_head(m, d, dtype):
    rows, H = 4 * m * max(1, 128 // m), 2
    for which in range(4):
        for bad in (float("nan"), float("inf")):
            x = _inputs(rows, H, d, dtype, which)
            perm = _perm(rows, rows, m)
            clean = bts.bt_ball_attention_backward(*x, perm, m)
            ball = rows // m // 2
            row = int(perm[ball * m + m // 2])
            x[which][row, 1, 3] = bad
            got = bts.bt_ball_attention_backward(*x, perm, m)
            inside = perm[ball * m:(ball + 1) * m].long()
            keep = torch.ones(rows, dtype=torch.bool, device="cuda")
            keep[inside] = False
            half = plain64.HALF[dtype]
            for a, b in zip(got, clean):
                assert torch.isfinite(a[keep]).all()
                assert torch.isfinite(a[:, 0]).all()
                # the same sums, perhaps in another order
                assert ((a[keep].double() - b[keep].double()).abs()
                        <= 4 * half * b[keep].double().abs() + 2e-2 * half * rows).all()
            assert not all(torch.isfinite(a[inside, 1]).all() for a in got)


def test_bad_perm_entry_is_recorded_not_read():
    for dtype, m in ((F32, 64), (BF16, 64), (BF16, 256)):
        x = _inputs(256, 2, 32, dtype, 12)
        perm = _perm(256, 256, 12)
        lost = int(perm[70])
        perm[70] = 10 ** 6
        out = tuple(torch.full_like(x[0], 7.0) for _ in range(3))
        got = bts.bt_ball_attention_backward(*x, perm, m, out=out)
        assert bts.bt_last_device_status() == 8  # BT_ERR_INTERNAL
        assert bts.bt_last_device_status() == 0
        perm[70] = -1
        want = bts.bt_ball_attention_backward(*x, perm, m)
        keep = torch.arange(256, device="cuda") != lost
        for a, b in zip(got, want):
            assert (a[lost] == 7.0).all() and torch.equal(a[keep], b[keep])


def test_gradient_of_the_forward_pass_by_differences():
    # float32 forward passes of the library: the change along a direction against the gradient
    rows, H, d, m = 128, 2, 32, 32
    x = _inputs(rows, H, d, F32, 21)
    perm = _perm(rows, rows, 21)
    grads = bts.bt_ball_attention_backward(*x, perm, m)
    t = 2.0 ** -7
    for i in range(3):
        dirn = _inputs(rows, H, d, F32, 30 + i)[0]
        f = []
        for s in (1, -1):
            y = [v.clone() for v in x[:3]]
            y[i] = y[i] + s * t * dirn
            f.append(float((bts.bt_ball_attention(*y, perm, m).double() * x[3].double()).sum()))
        want = float((grads[i].double() * dirn.double()).sum())
        # curvature t^2 / 6 times third derivatives of order the sum itself, and float rounding of O over 2 t
        assert abs((f[0] - f[1]) / (2 * t) - want) <= 1e-2 * float((grads[i] * dirn).double().abs().sum()) ** 0.5 + 0.05


def test_equal_calls_and_streams_give_equal_bits():
    for dtype, m, d in ((BF16, 128, 32), (BF16, 32, 64), (F32, 64, 32)):
        x = _inputs(4096, 4, d, dtype, 40)
        perm = _perm(4000, 4096, 1)
        want = bts.bt_ball_attention_backward(*x, perm, m)
        torch.cuda.synchronize()
        ss = [torch.cuda.Stream() for _ in range(2)]
        got = [bts.bt_ball_attention_backward(*x, perm, m, stream=s) for s in ss for _ in range(2)]
        torch.cuda.synchronize()
        for o in got:
            for a, b in zip(o, want):
                assert torch.equal(a[perm[perm >= 0].long()], b[perm[perm >= 0].long()])


def test_captured_and_replayed():
    x = _inputs(2048, 4, 32, BF16, 50)
    perm = _perm(2048, 2048, 2)
    out = tuple(torch.zeros_like(x[0]) for _ in range(3))
    bts.bt_ball_attention_backward(*x, perm, 128, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        bts.bt_ball_attention_backward(*x, perm, 128, out=out)
    y = _inputs(2048, 4, 32, BF16, 51)
    for a, b in zip(x, y):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, bts.bt_ball_attention_backward(*y, perm, 128)):
        assert torch.equal(a, b)


def test_tree_of_a_ragged_batch():
    wl = workloads.ragged(batch=3, n_min=200, n_max=3000)
    perm, _ = bts.bt_build_segmented(torch.from_numpy(wl.coords).cuda(), wl.offsets, 64)
    for dtype in (BF16, F32):
        _check(_inputs(len(wl.coords), 2, 32, dtype, 60), perm, 64)


def test_refusals():
    x = _inputs(128, 2, 32, BF16, 70)
    perm = _perm(128, 128, 3)
    call = bts.bt_ball_attention_backward
    with pytest.raises(ValueError):
        call(x[0], x[1][:64], x[2], x[3], perm, 32)
    with pytest.raises(TypeError):
        call(x[0], x[1].float(), x[2], x[3], perm, 32)
    with pytest.raises(TypeError):
        call(*(t.half() for t in x), perm, 32)
    with pytest.raises(TypeError):
        call(*x, perm.long(), 32)
    with pytest.raises(ValueError):
        call(*x, perm.cpu(), 32)
    with pytest.raises(ValueError):
        call(*x, perm, 32, npad=256)
    with pytest.raises(ValueError):
        call(*x, perm, 32, out=(x[0], torch.empty_like(x[0]), torch.empty_like(x[0])))
    with pytest.raises(ValueError):
        call(x[0].transpose(0, 1).contiguous().transpose(0, 1), *x[1:], perm, 32)
    for m, d in ((0, 32), (257, 32), (48, 32)):
        with pytest.raises(bts.BtsError) as e:
            call(*x, perm, m)
        assert e.value.status == "BT_ERR_SHAPE"
    with pytest.raises(bts.BtsError) as e:
        call(*(torch.zeros(128, 2, 48, dtype=BF16, device="cuda"),) * 4, perm, 32)
    assert e.value.status == "BT_ERR_SHAPE"
    flat = torch.zeros(128 * 64 + 1, dtype=BF16, device="cuda")
    with pytest.raises(bts.BtsError) as e:
        call(flat[1:].view(128, 2, 32), *x[1:], perm, 32)  # not 16-byte aligned
    assert e.value.status == "BT_ERR_ARG"
