"""What a call makes and gives back itself belongs to the stream that uses it.

The work is held back on a side stream; an array that the current stream allocates meanwhile must not share the memory
of the call's inverse, or of its workspace.
"""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16 = torch.bfloat16


def _held_back(call, sizes):
    """call(stream=...) on a side stream that is still busy, while the current stream fills arrays of the given sizes."""
    def fill():
        return [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)  # so that nothing below asks the driver for memory
    fill()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(60_000_000)
    got = call(side)
    mine = fill()
    assert not side.query()  # the work is still to come
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in mine)
    assert bts.bt_last_device_status(side) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def _features(rows, C, H, d):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, C, generator=g, device="cuda").to(BF16)
    wt = (torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5).to(BF16)
    return x, wt, torch.randperm(rows, generator=g, device="cuda").to(torch.int32)


def test_inverse_of_the_projection():
    rows, C, H, d = 1 << 19, 64, 2, 32
    x, wt, perm = _features(rows, C, H, d)
    out = tuple(torch.empty((rows, H, d), dtype=BF16, device="cuda") for _ in range(3))

    def call(stream):
        bts.bt_qkv_project(x, wt, H, d, perm=perm, out=out, stream=stream)
        return out if stream else [t.clone() for t in out]
    _held_back(call, [4 * rows])


def test_workspace_of_the_layer():
    rows, C, H, d, m = 1 << 16, 64, 2, 32, 128
    x, wt, perm = _features(rows, C, H, d)
    O = torch.empty((rows, H, d), dtype=BF16, device="cuda")

    def call(stream):
        bts.bt_projected_ball_attention(x, perm, wt, m, H, d, out=O, stream=stream)
        return [O if stream else O.clone()]
    _held_back(call, [bts.bt_projected_workspace_size(rows, rows, H, d, BF16)])


def test_workspace_of_a_build():
    n, m = 1 << 16, 128
    pts = torch.from_numpy(workloads.uniform_cloud(n, 3)).cuda()
    perm = torch.empty(n, dtype=torch.int32, device="cuda")

    def call(stream):
        bts.bt_build(pts, m, perm=perm, stream=stream)
        return [perm if stream else perm.clone()]
    _held_back(call, [bts.bt_build_workspace_size([0, n], m)])
