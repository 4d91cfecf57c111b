"""The roundings of the 8-bit projection, one by one: the exact sum as a float, times the row's scale, times the
channel's, then the result's type.  Every kernel gives these bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,C,H,d", [(7, 256, 2, 32), (7, 8000, 2, 32), (300, 256, 2, 32), (300, 8192, 2, 32),
                                        (300, 6001, 2, 32), (300, 256, 3, 3), (300, 8000, 3, 3)])
def test_bits(rows, C, H, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + C)

    def ints(n):
        # a row's values have the mean 62.75, so that a sum's is 3,938 C: 23.6 million and more from C = 6,001 on, above
        # 2^24, and 1 million at C = 256, below
        q = torch.randint(-127, 128, (n, C), generator=g, device="cuda") // 2 + 63
        return q.to(torch.int8), torch.exp(torch.randn(n, generator=g, device="cuda"))
    (xq, xs), (wq, ws) = ints(rows), ints(3 * H * d)
    exact = xq.double() @ wq.double().T
    assert (exact.abs().max() > 2 ** 24) == (C >= 6001)
    want = (exact.float() * xs[:, None] * ws[None, :]).to(dtype)
    got = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype)
    assert torch.equal(torch.stack(got, 1).reshape(rows, 3 * H * d), want)
