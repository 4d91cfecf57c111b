"""Layers over slot maps that do not name every row, against their steps in the original row order.

A layer's slot-order path (bf16, d = 32, an even number of heads, balls of 16 to 128) and its gathering path compute the
same numbers: the projection's rows do not depend on where they are stored, and the attention sees the same tiles.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(BF16, 32, 2), (F32, 32, 2), (BF16, 64, 2), (BF16, 32, 3)]  # the first takes the slot-order path


def _inputs(rows, C, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn(rows, C, generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    wq, ws = bts.bt_quantize_i8(torch.randn(3 * H * d, C, generator=g, device="cuda") / C ** 0.5)
    return x, r, gamma, wq, ws, torch.randperm(rows, generator=g, device="cuda").to(torch.int32)


def _steps(x, r, gamma, wq, ws, perm, m, H, d, dtype, npad, out):
    xq, xs, h = bts.bt_rms_norm_i8(x, gamma, residual=r)
    q, k, v = bts.bt_qkv_project_i8(xq, xs, wq, ws, H, d, dtype=dtype)
    return bts.bt_ball_attention(q, k, v, perm, m, npad=npad, out=out), h


@pytest.mark.parametrize("dtype,d,H", SHAPES)
def test_fewer_slots_than_rows(dtype, d, H):
    rows, C, m = 700, 64, 32
    x, r, gamma, wq, ws, perm = _inputs(rows, C, H, d, dtype, 1)
    for p, npad in ((perm, 512), (perm[:384].contiguous(), None), (torch.cat((perm[:250], perm.new_full((6,), -1))), 256)):
        out = torch.full((rows, H, d), 7.0, dtype=dtype, device="cuda")
        O, h = _steps(x, r, gamma, wq, ws, p, m, H, d, dtype, npad, out)
        stream = x.clone()  # the stream is updated in place, and once
        got = torch.full((rows, H, d), 7.0, dtype=dtype, device="cuda")
        bts.bt_projected_ball_attention_i8(stream, p, wq, ws, m, H, d, weight=gamma, residual=r, hout=stream, out=got,
                                           npad=npad)
        assert bts.bt_last_device_status() == 0
        assert torch.equal(stream, h)
        assert torch.equal(got, O)


@pytest.mark.parametrize("dtype,d,H", SHAPES)
def test_fewer_slots_than_rows_in_16_and_32_bits(dtype, d, H):
    rows, C, m = 700, 64, 32
    x, _, _, wq, ws, perm = _inputs(rows, C, H, d, dtype, 3)
    wt = (wq.float() * ws[:, None]).to(dtype)
    for p, npad in ((perm, 512), (perm[:384].contiguous(), None)):
        want, got = (torch.full((rows, H, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        bts.bt_ball_attention(*bts.bt_qkv_project(x, wt, H, d), p, m, npad=npad, out=want)
        bts.bt_projected_ball_attention(x, p, wt, m, H, d, out=got, npad=npad)
        assert bts.bt_last_device_status() == 0
        assert torch.equal(got, want)


def test_a_refused_call_leaves_the_stream_alone():
    # whatever a later step would refuse is refused before the residual is added
    rows, C, H, d, m = 256, 64, 2, 32, 32
    x, r, gamma, wq, ws, perm = _inputs(rows, C, H, d, BF16, 2)
    nb = bts.bt_projected_i8_workspace_size(rows, rows, C, H, d, BF16)
    work = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.empty(rows, H, d, dtype=BF16, device="cuda")
    raw = torch.zeros(4 * rows + 4, dtype=torch.uint8, device="cuda")

    def call(perm=perm.data_ptr(), ws=ws.data_ptr(), wq=wq.data_ptr()):
        return bts._lib.bt_projected_ball_attention_i8(x.data_ptr(), r.data_ptr(), gamma.data_ptr(), 1e-6, perm, rows,
                                                       rows, C, wq, ws, m, H, d, 1, x.data_ptr(), out.data_ptr(),
                                                       work.data_ptr(), nb, None)
    before = x.clone()
    for kw in ({"perm": raw.data_ptr() + 2}, {"ws": raw.data_ptr() + 1}, {"ws": None}, {"wq": None}):
        assert call(**kw) == 1  # BT_ERR_ARG
        torch.cuda.synchronize()
        assert torch.equal(x, before)
    assert call() == 0
    torch.cuda.synchronize()
    assert not torch.equal(x, before)
