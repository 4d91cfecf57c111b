"""Results that the training and 8-bit calls allocate, in rows that no slot names."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _fill_the_allocator(*shapes):
    """Leaves memory of the given sizes full of NaN to the next allocations."""
    t = [torch.full(s, float("nan"), device="cuda") for s in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("side", [False, True])
def test_gradients_of_rows_without_a_slot_are_zero(dtype, side):
    rows, H, d, m = 300, 2, 32, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    x = [torch.randn(rows, H, d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    perm = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    stream = torch.cuda.Stream() if side else None
    cases = [(perm[:256].contiguous(), None),                             # fewer slots than rows
             (torch.cat((perm, perm.new_full((20,), -1))), 160),          # a part of a tree's slots
             (None, 288),                                                 # the first rows alone
             (perm[:0].contiguous(), None), (None, 0)]                    # no slot at all
    for p, npad in cases:
        n = npad if npad is not None else p.numel()
        named = torch.zeros(rows, dtype=torch.bool, device="cuda")
        slots = torch.arange(n, device="cuda") if p is None else p[:n].long()
        named[slots[slots >= 0]] = True
        torch.cuda.synchronize()
        if side:
            with torch.cuda.stream(stream):
                _fill_the_allocator((rows, H, d))
        else:
            _fill_the_allocator((rows, H, d))
        got = bts.bt_ball_attention_backward(*x, p, m, npad=npad, stream=stream)
        torch.cuda.synchronize()
        out = tuple(torch.zeros_like(x[0]) for _ in range(3))
        bts.bt_ball_attention_backward(*x, p, m, npad=npad, out=out)
        for a, b in zip(got, out):
            assert (a[~named] == 0).all()
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_output_of_rows_without_a_slot_is_zero(dtype):
    rows, C, H, d, m = 300, 64, 2, 32, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, C, generator=g, device="cuda").to(dtype)
    wq, ws = bts.bt_quantize_i8(torch.randn(3 * H * d, C, generator=g, device="cuda"))
    _fill_the_allocator((rows, H, d))
    O, _ = bts.bt_projected_ball_attention_i8(x, None, wq, ws, m, H, d, npad=288)
    assert (O[288:] == 0).all() and torch.isfinite(O).all()
    _fill_the_allocator((rows, H, d))
    O, _ = bts.bt_projected_ball_attention_i8(x, torch.empty(0, dtype=torch.int32, device="cuda"), wq, ws, m, H, d)
    assert (O == 0).all()
