"""What the norm returns where it writes over its input."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_over_its_input_has_no_stream_to_return(dtype):
    # without a residual h is X; where Y takes X's place it is gone, and must not be taken for the backward pass's input
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(50, 96, generator=g, device="cuda").to(dtype)
    r = torch.randn(50, 96, generator=g, device="cuda").to(dtype)
    want, h = bts.bt_rms_norm(x)
    assert h is x
    for view in (False, True):
        x2 = x.clone()
        y, h = bts.bt_rms_norm(x2, out=x2.view(50, 96) if view else x2)
        assert h is None
        assert torch.equal(y, want) and torch.equal(x2, want)
    x2 = x.clone()  # with a residual h has memory of its own
    want, hw = bts.bt_rms_norm(x, residual=r)
    y, h = bts.bt_rms_norm(x2, residual=r, out=x2)
    assert torch.equal(y, want) and torch.equal(h, hw)
