"""Attention's backward pass where finite inputs give scores that float cannot hold.

Two rows of values of 1e20 have the product 1e40 d, which is infinite in float, and the softmax of a row with an
infinite maximum is NaN.  That ball and head lose their gradients; every other ball's, and the other head's, equal those
of a call without such values bit by bit: a weight of 0 adds 0 to a sum of finite products.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,d", [(1, 32), (2, 64), (4, 32), (4, 64), (7, 32), (16, 32), (16, 64), (32, 32), (64, 64),
                                 (128, 32), (200, 32)])
def test_scores_beyond_float_stay_in_their_ball_and_head(m, d, dtype):
    balls, H = max(4, 160 // m), 2
    rows = balls * m
    g = torch.Generator(device="cuda").manual_seed(m + d)
    x = [torch.randn(rows, H, d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    clean = bts.bt_ball_attention_backward(*x, perm, m)
    inside = perm[m:2 * m].long()  # the second ball
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[inside] = False
    for sign in (1.0, -1.0):
        y = [t.clone() for t in x]
        y[0][inside[0], 1] = 1e20
        y[1][inside, 1] = sign * 1e20
        assert all(torch.isfinite(t).all() for t in y)
        got = bts.bt_ball_attention_backward(*y, perm, m)
        assert bts.bt_last_device_status() == 0
        for a, b in zip(got, clean):
            assert torch.equal(a[keep], b[keep])
            assert torch.equal(a[:, 0], b[:, 0])
        assert not all(torch.isfinite(a[inside, 1]).all() for a in got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m", [4, 16, 64, 128])
def test_weights_gradients_beyond_float_stay_in_their_ball_and_head(m, dtype):
    # dO and V whose product is infinite: dP and delta of one row
    rows, H, d = 4 * m * max(1, 64 // m), 2, 32
    g = torch.Generator(device="cuda").manual_seed(m)
    x = [torch.randn(rows, H, d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    clean = bts.bt_ball_attention_backward(*x, perm, m)
    inside = perm[m:2 * m].long()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[inside] = False
    x[2][inside, 1] = 1e20
    x[3][inside[0], 1] = 1e20
    got = bts.bt_ball_attention_backward(*x, perm, m)
    assert bts.bt_last_device_status() == 0
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
        assert torch.equal(a[:, 0], b[:, 0])
