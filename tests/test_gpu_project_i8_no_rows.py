"""The 8-bit projection of no rows into slots: every slot is a dummy, with or without an inverse."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("given", [False, True])
def test_dummies_alone(dtype, given):
    xq, xs = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    wq, ws = torch.ones(192, 64, dtype=torch.int8, device="cuda"), torch.ones(192, device="cuda")
    perm = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    inv = torch.empty(0, dtype=torch.int32, device="cuda") if given else None
    out = tuple(torch.full((256, 2, 32), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    got = bts.bt_qkv_project_i8(xq, xs, wq, ws, 2, 32, dtype=dtype, perm=perm, inv=inv, out=out)
    assert bts.bt_last_device_status() == 0
    assert all((t == 0).all() for t in got)
