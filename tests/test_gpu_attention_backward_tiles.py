"""Attention's backward pass where a CTA walks several tiles, and shapes beside those of test_gpu_attention_backward.

The float64 formula is evaluated with torch on the GPU, ball by ball in batches, with the bounds that
plain64.attention_backward derives: P and dS are rounded once to bf16 (2^-8) on the tensor cores, results to bf16, and
float sums of n terms are off by (n + 2) 2^-24 of the absolute terms.
"""
import math

import pytest
import torch

from plain64 import HALF, U

pytestmark = pytest.mark.gpu

bts = pytest.importorskip("ball_tree_sparse_b200")

BF16, F32 = torch.bfloat16, torch.float32


def _formula(x, perm, m, half):
    """(gradients, bounds) as float64 [rows, H, d], for a perm without dummies."""
    d = x[0].shape[2]
    sc = 1 / math.sqrt(d)
    grads = [torch.zeros_like(x[0], dtype=torch.float64) for _ in range(3)]
    bounds = [torch.zeros_like(x[0], dtype=torch.float64) for _ in range(3)]
    balls = perm.long().view(-1, m)
    for idx in balls.split(max(1, (1 << 22) // (m * m * x[0].shape[1]))):
        q, k, v, g = (t[idx].double().transpose(1, 2) for t in x)  # [balls, H, m, d]
        s = q @ k.transpose(2, 3) * sc
        p = torch.softmax(s, 3)
        dp = g @ v.transpose(2, 3)
        delta = (p * dp).sum(3, keepdim=True)
        ds = p * (dp - delta)
        es = (d + 4) * U * (q.abs() @ k.abs().transpose(2, 3)) * sc + 4 * U * s.abs()
        ep = 2 * es.amax(3, keepdim=True) + (m + 16) * U
        eg = (d + 2) * U * (g.abs() @ v.abs().transpose(2, 3))
        ed = (p * (ep * dp.abs() + eg)).sum(3, keepdim=True) + (m + 4) * U * (p * dp.abs()).sum(3, keepdim=True)
        eds = p * (ep * (dp - delta).abs() + eg + ed + 4 * U * (dp.abs() + delta.abs())) + half * ds.abs()
        pt, dst = p.transpose(2, 3), ds.transpose(2, 3)
        out = (ds @ k * sc, dst @ q * sc, pt @ g)
        err = (sc * (eds @ k.abs() + (m + 4) * U * (ds.abs() @ k.abs())),
               sc * (eds.transpose(2, 3) @ q.abs() + (m + 4) * U * (dst.abs() @ q.abs())),
               ((ep + half) * p).transpose(2, 3) @ g.abs() + (m + 2) * U * (pt @ g.abs()))
        for o, b, t, e in zip(grads, bounds, out, err):
            o[idx] = t.transpose(1, 2)
            b[idx] = (1.01 * e + 1.01 * HALF[x[0].dtype] * t.abs() + 1e-37).transpose(1, 2)
    return grads, bounds


def _inputs(rows, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(rows, H, d, generator=g, device="cuda").to(dtype) for _ in range(4)]


@pytest.mark.parametrize("m,d,H", [(128, 32, 4), (128, 64, 3), (64, 32, 3), (64, 64, 2), (32, 64, 5), (16, 32, 1),
                                   (100, 32, 3), (65, 64, 2)])
def test_many_tiles(m, d, H):
    rows = 128 // m * m * 700
    x = _inputs(rows, H, d, BF16, m + d)
    perm = torch.randperm(rows, generator=torch.Generator(device="cuda").manual_seed(m), device="cuda").to(torch.int32)
    got = bts.bt_ball_attention_backward(*x, perm, m)
    assert bts.bt_last_device_status() == 0
    for a, b, e in zip(got, *_formula(x, perm, m, HALF[BF16])):
        over = (a.double() - b).abs() - e
        assert (over <= 0).all(), float(over.max())


@pytest.mark.parametrize("m,d", [(128, 32), (128, 64), (90, 32), (66, 64)])
def test_one_ball_with_dummies_and_values_not_finite(m, d):
    # a tile that is one ball: dummies in any slot, and a ball whose values are not finite next to clean ones
    balls, H = 40, 2
    perm = torch.full((balls * m,), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(m)
    slots = torch.randperm(balls * m, generator=g, device="cuda")[:balls * m * 3 // 4]
    rows = slots.numel()
    perm[slots] = torch.arange(rows, dtype=torch.int32, device="cuda")
    x = _inputs(rows, H, d, BF16, 5)
    clean = bts.bt_ball_attention_backward(*x, perm, m)
    assert bts.bt_last_device_status() == 0
    inside = perm[7 * m:8 * m]
    inside = inside[inside >= 0].long()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[inside] = False
    for which in range(4):
        for bad in (float("nan"), float("inf"), float("-inf")):
            y = [t.clone() for t in x]
            y[which][inside[3], 1, 5] = bad
            got = bts.bt_ball_attention_backward(*y, perm, m)
            assert bts.bt_last_device_status() == 0
            for a, b in zip(got, clean):
                assert torch.equal(a[keep], b[keep]) and torch.equal(a[:, 0], b[:, 0])
            assert not all(torch.isfinite(a[inside, 1]).all() for a in got)


def test_dummy_balls_between_real_ones():
    # whole tiles of dummies are skipped, by groups that take items of their own too
    for d, H in ((32, 3), (64, 5)):
        m, tiles = 128, 900
        live = torch.rand(tiles, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda") < 0.4
        rows = int(live.sum()) * m
        perm = torch.full((tiles, m), -1, dtype=torch.int32, device="cuda")
        perm[live] = torch.randperm(rows, generator=torch.Generator(device="cuda").manual_seed(1),
                                    device="cuda").to(torch.int32).view(-1, m)
        x = _inputs(rows, H, d, BF16, 9)
        got = bts.bt_ball_attention_backward(*x, perm.flatten(), m)
        want = bts.bt_ball_attention_backward(*x, perm[live].flatten().contiguous(), m)
        assert bts.bt_last_device_status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    jobs = []
    for i, (m, d) in enumerate(((128, 32), (64, 64), (128, 64), (32, 32))):
        rows = 128 * 200
        x = _inputs(rows, 2, d, BF16, 20 + i)
        perm = torch.randperm(rows, device="cuda").to(torch.int32)
        jobs.append((x, perm, m, bts.bt_ball_attention_backward(*x, perm, m), torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = [[bts.bt_ball_attention_backward(*x, perm, m, stream=s) for _ in range(3)] for x, perm, m, _, s in jobs]
    torch.cuda.synchronize()
    for (_, _, _, want, s), runs in zip(jobs, out):
        assert bts.bt_last_device_status(s) == 0
        for got in runs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
