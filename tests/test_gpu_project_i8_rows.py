"""The 8-bit projection of rows that no tensor map takes: any length and any address, between bytes that must not count.

The bounds are those of test_gpu_project_i8: an exact sum, three roundings of float, half a step of the type.
"""
import pytest
import torch

import plain64
from plain64 import HALF, U

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _inside(rows, C, offset, seed):
    """int8 [rows, C] at any address, between bytes of 127."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole = torch.full((64 + rows * C + 64,), 127, dtype=torch.int8, device="cuda")
    q = whole[32 + offset:32 + offset + rows * C].view(rows, C)
    q.copy_(torch.randint(-127, 128, (rows, C), generator=g, device="cuda"))
    return q, torch.rand(rows, generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C", [(33, 1), (40, 2), (129, 3), (128, 5), (200, 15), (257, 17), (300, 127), (300, 129),
                                    (1000, 130), (513, 255), (140, 1023), (600, 1300)])
def test_any_length_and_address(rows, C, dtype):
    H, d = 3, 16
    for ox, ow in ((0, 0), (1, 2), (3, 1)):
        (x, xs), (w, ws) = _inside(rows, C, ox, C), _inside(3 * H * d, C, ow, C + 1)
        got = bts.bt_qkv_project_i8(x, xs, w, ws, H, d, dtype=dtype)
        assert bts.bt_last_device_status() == 0
        want = plain64.project_i8(x, xs, w, ws)
        for t, a in enumerate(got):
            y = want[:, t * H * d:(t + 1) * H * d].reshape(rows, H, d)
            plain64.within(a, y, 1.01 * (3 * U + (HALF[dtype] if dtype == BF16 else 0)) * y.abs() + 1e-38)


def test_many_tiles_in_tree_order():
    # several tiles a CTA, dummies between the slots, both loaders
    rows, H, d = 70000, 4, 32
    npad = 81920
    g = torch.Generator(device="cuda").manual_seed(3)
    perm = torch.full((npad,), -1, dtype=torch.int32, device="cuda")
    slots = torch.randperm(npad, generator=g, device="cuda")[:rows]
    perm[slots] = torch.arange(rows, dtype=torch.int32, device="cuda")
    for C in (128, 99):
        (x, xs), (w, ws) = _inside(rows, C, 0, 1), _inside(3 * H * d, C, 0, 2)
        tree = bts.bt_qkv_project_i8(x, xs, w, ws, H, d, perm=perm)
        plain = bts.bt_qkv_project_i8(x, xs, w, ws, H, d)
        assert bts.bt_last_device_status() == 0
        for a, b in zip(tree, plain):
            assert torch.equal(a[slots], b)
            assert (a[perm < 0] == 0).all()
        want = plain64.project_i8(x[:500], xs[:500], w, ws)[:, :H * d].reshape(500, H, d)
        plain64.within(plain[0][:500], want, 1.01 * (3 * U + HALF[BF16]) * want.abs() + 1e-38)


def test_what_a_call_allocates_belongs_to_its_stream():
    # the inverse of perm that the call makes is given back to the stream that uses it: an array that the current stream
    # allocates while the work is still to come must not share its memory
    rows, C, H, d = 1 << 20, 16, 1, 8
    (x, xs), (w, ws) = _inside(rows, C, 0, 1), _inside(3 * H * d, C, 0, 2)
    perm = torch.arange(rows, dtype=torch.int32, device="cuda")
    want = bts.bt_qkv_project_i8(x, xs, w, ws, H, d, perm=perm)
    side = torch.cuda.Stream()

    def fill():
        return [torch.full((rows,), 7, dtype=torch.int32, device="cuda") for _ in range(16)]
    bts.bt_qkv_project_i8(x, xs, w, ws, H, d, perm=perm, stream=side)  # so that nothing below asks the driver for memory
    fill()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    got = bts.bt_qkv_project_i8(x, xs, w, ws, H, d, perm=perm, stream=side)
    mine = fill()
    assert not side.query()  # the work is still to come
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in mine)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
