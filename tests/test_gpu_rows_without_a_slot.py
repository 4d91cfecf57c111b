"""Slot maps that leave rows without a slot, in the calls that make the inverse themselves.

The inverse lies in memory that held something else before: another call's inverse in a workspace, any values in a new
tensor.  Whatever was there, a row that no slot names is stored nowhere, and the result equals that of the original
order, in which no inverse is needed.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _map(rows, npad, named, seed):
    """`named` of the rows in random slots of npad."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.full((npad,), -1, dtype=torch.int32, device="cuda")
    slots = torch.randperm(npad, generator=g, device="cuda")[:named]
    perm[slots] = torch.randperm(rows, generator=g, device="cuda")[:named].to(torch.int32)
    return perm


def _features(rows, C, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, C, generator=g, device="cuda").to(dtype)
    return x, torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5


def _stale(rows):
    """Leaves inverses (every entry a slot) to the allocations that follow."""
    t = [torch.randint(0, rows, (rows,), dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del t


def _expect(plain, perm):
    real = perm >= 0
    out = plain[perm.clamp(min=0).long()]
    return torch.where(real[:, None, None], out, torch.zeros_like(out))


@pytest.mark.parametrize("rows,npad,named", [(30, 64, 20), (700, 1024, 500), (1024, 1024, 1000), (5000, 8192, 1),
                                             (3000, 4096, 0)])
def test_projections(rows, npad, named):
    H, d = 2, 32
    for C, dtype in ((64, BF16), (64, F32), (99, BF16)):
        x, wt = _features(rows, C, H, d, dtype, rows)
        (xq, xs), (wq, ws) = bts.bt_quantize_i8(x), bts.bt_quantize_i8(wt)
        plain8 = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype)
        plain = bts.bt_qkv_project(x, wt.to(dtype), H, d)
        for seed in range(4):
            perm = _map(rows, npad, named, seed)
            _stale(rows)
            got8 = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype, perm=perm)
            _stale(rows)
            got = bts.bt_qkv_project(x, wt.to(dtype), H, d, perm=perm)
            assert bts.bt_last_device_status() == 0
            for a, b in zip((*got8, *got), (*plain8, *plain)):
                assert torch.equal(a, _expect(b, perm))


@pytest.mark.parametrize("m", [16, 128])
def test_layers_after_another_call_in_the_same_workspace(m):
    rows, npad, C, H, d = 900, 1024, 64, 4, 32
    x, wt = _features(rows, C, H, d, BF16, 5)
    wq, ws = bts.bt_quantize_i8(wt)
    work = torch.empty(bts.bt_projected_i8_workspace_size(npad, rows, C, H, d, BF16), dtype=torch.uint8, device="cuda")
    work16 = torch.empty(bts.bt_projected_workspace_size(npad, rows, H, d, BF16), dtype=torch.uint8, device="cuda")
    xq, xs, _ = bts.bt_rms_norm_i8(x)
    qkv8 = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d)
    qkv = bts.bt_qkv_project(x, wt.to(BF16), H, d)
    for seed in range(4):
        whole, part = _map(rows, npad, rows, 10 + seed), _map(rows, npad, 600, seed)
        for perm in (whole, part, part):
            want8, want, got8, got = (torch.full((rows, H, d), 7.0, dtype=BF16, device="cuda") for _ in range(4))
            bts.bt_ball_attention(*qkv8, perm, m, out=want8)
            bts.bt_ball_attention(*qkv, perm, m, out=want)
            bts.bt_projected_ball_attention_i8(x, perm, wq, ws, m, H, d, out=got8, work=work)
            bts.bt_projected_ball_attention(x, perm, wt.to(BF16), m, H, d, out=got, ws=work16)
            assert bts.bt_last_device_status() == 0
            assert torch.equal(got8, want8) and torch.equal(got, want)


def test_an_inverse_of_the_caller_says_so_too():
    rows, C, H, d = 200, 64, 2, 32
    x, wt = _features(rows, C, H, d, BF16, 6)
    (xq, xs), (wq, ws) = bts.bt_quantize_i8(x), bts.bt_quantize_i8(wt)
    perm = _map(rows, 256, 150, 7)
    inv = torch.full((rows,), bts.BT_NO_SLOT, dtype=torch.int32, device="cuda")
    bts.bt_invert_perm(perm, rows, inv)
    got = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, perm=perm, inv=inv)
    assert bts.bt_last_device_status() == 0
    for a, b in zip(got, bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d)):
        assert torch.equal(a, _expect(b, perm))
    inv[perm[perm >= 0][0].long()] = -1  # no slot, and does not say so
    bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, perm=perm, inv=inv)
    assert bts.bt_last_device_status() == 8 and bts.bt_last_device_status() == 0
