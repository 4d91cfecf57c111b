"""Slot maps with entries that are no rows, in the calls that invert them: recorded, never written through.

A slot with such an entry is a dummy: the result is that of the map with -1 in its place.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32
BAD = (0, 1, 300, 2 ** 30, 2 ** 31 - 1)  # beyond the number of rows


def _status_is_internal():
    assert bts.bt_last_device_status() == 8  # BT_ERR_INTERNAL
    assert bts.bt_last_device_status() == 0


def _maps(rows, npad, seed):
    """A map of every row, with some entries out of range, and the same with those as dummies."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.full((npad,), -1, dtype=torch.int32, device="cuda")
    slots = torch.randperm(npad, generator=g, device="cuda")
    perm[slots[:rows]] = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    at = torch.cat((slots[:3], slots[-2:]))  # rows lose their slots; dummies
    bad, good = perm.clone(), perm.clone()
    bad[at] = torch.tensor([min(rows + b, 2 ** 31 - 1) for b in BAD], dtype=torch.int32, device="cuda")
    good[at] = -1
    return bad, good


def test_inverse():
    for rows, npad in ((1, 8), (100, 128), (5000, 8192)):
        whole = torch.full((rows + 2048,), 7, dtype=torch.int32, device="cuda")
        inv = whole[1024:1024 + rows]
        inv.fill_(bts.BT_NO_SLOT)
        bad, good = _maps(rows, npad, rows)
        bts.bt_invert_perm(bad, rows, inv)
        _status_is_internal()
        want = torch.full((rows,), bts.BT_NO_SLOT, dtype=torch.int32, device="cuda")
        bts.bt_invert_perm(good, rows, want)
        assert bts.bt_last_device_status() == 0
        assert torch.equal(inv, want)
        assert (whole[:1024] == 7).all() and (whole[1024 + rows:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,npad,C", [(20, 64, 64), (300, 512, 64), (300, 512, 99), (3000, 4096, 128)])
def test_projections(rows, npad, C, dtype):
    H, d = 2, 32
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, C, generator=g, device="cuda").to(dtype)
    wt = torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5
    (xq, xs), (wq, ws) = bts.bt_quantize_i8(x), bts.bt_quantize_i8(wt)
    bad, good = _maps(rows, npad, C)
    inv = torch.full((rows,), bts.BT_NO_SLOT, dtype=torch.int32, device="cuda")
    bts.bt_invert_perm(good, rows, inv)
    for given in (None, inv):
        for call in (lambda p, o: bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype, perm=p, inv=given, out=o),
                     lambda p, o: bts.bt_qkv_project(x, wt.to(dtype), H, d, perm=p, inv=given, out=o)):
            got, want = (tuple(torch.full((npad, H, d), v, dtype=dtype, device="cuda") for _ in range(3))
                         for v in (float("nan"), 7.0))
            call(bad, got)
            _status_is_internal()
            call(good, want)
            assert bts.bt_last_device_status() == 0
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d,H", [(BF16, 32, 2), (F32, 32, 2), (BF16, 64, 2), (BF16, 32, 3)])
@pytest.mark.parametrize("m", [32, 128])
def test_layers(m, dtype, d, H):
    rows, npad, C = 900, 1024, 64
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(rows, C, generator=g, device="cuda").to(dtype)
    wt = torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5
    wq, ws = bts.bt_quantize_i8(wt)
    sizes = (bts.bt_projected_i8_workspace_size(npad, rows, C, H, d, dtype),
             bts.bt_projected_workspace_size(npad, rows, H, d, dtype))
    calls = (lambda p, o, w: bts.bt_projected_ball_attention_i8(x, p, wq, ws, m, H, d, out=o, work=w),
             lambda p, o, w: bts.bt_projected_ball_attention(x, p, wt.to(dtype), m, H, d, out=o, ws=w))
    bad, good = _maps(rows, npad, m)
    for call, n in zip(calls, sizes):
        whole = torch.full((n + 8192,), 0xFF, dtype=torch.uint8, device="cuda")  # floats and 16-bit values of it are NaN
        got, want = (torch.full((rows, H, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        call(bad, got, whole[4096:4096 + n])
        _status_is_internal()
        assert (whole[:4096] == 0xFF).all() and (whole[4096 + n:] == 0xFF).all()
        call(good, want, whole[4096:4096 + n])
        assert bts.bt_last_device_status() == 0
        assert torch.equal(got, want)
