"""CPU checks of the training and 8-bit calls: argument errors come back before any launch, workspace sizes."""
import ctypes

import pytest

P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
one, odd = ctypes.c_void_p(256), ctypes.c_void_p(257)
ARG, SHAPE, WORKSPACE, UNSUPPORTED = 1, 2, 4, 7
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def b():
    return pytest.importorskip("ball_tree_sparse_b200")


def test_attention_backward(b):
    def call(Q=one, K=one, V=one, dO=one, perm=one, npad=128, rows=128, m=32, H=2, d=32, dt=BF16, dQ=one, dK=one,
             dV=one):
        return b._lib.bt_ball_attention_backward(Q, K, V, dO, perm, npad, rows, m, H, d, dt, dQ, dK, dV, None)
    for n in ("Q", "K", "V", "dO", "dQ", "dK", "dV"):
        assert call(**{n: None}) == ARG
        assert call(**{n: ctypes.c_void_p(264)}) == ARG  # 8-byte aligned
    assert call(npad=-32) == ARG and call(rows=-1) == ARG and call(H=0) == ARG and call(dt=2) == ARG
    assert call(perm=None, rows=127) == ARG  # slots without rows
    assert call(perm=ctypes.c_void_p(258)) == ARG
    for kw in ({"m": 0}, {"m": 257}, {"d": 48}, {"d": 128}, {"npad": 100}):
        assert call(**kw) == SHAPE
    assert call(rows=2 ** 31 - 1) == UNSUPPORTED and call(npad=2 ** 31) == UNSUPPORTED and call(H=65536) == UNSUPPORTED
    assert call(npad=0) == 0 and call(rows=0) == 0 and call(npad=0, Q=None, dV=None) == 0


def test_norm(b):
    def call(X=one, R=one, w=one, rows=4, C=64, eps=1e-6, dt=BF16, H=one, Y=one):
        return b._lib.bt_rms_norm(X, R, w, rows, C, eps, dt, H, Y, None)

    def call8(X=one, R=one, w=one, rows=4, C=64, eps=1e-6, dt=BF16, H=one, Y=one, s=one):
        return b._lib.bt_rms_norm_i8(X, R, w, rows, C, eps, dt, H, Y, s, None)
    for f in (call, call8):
        assert f(X=None) == ARG and f(Y=None) == ARG and f(rows=-1) == ARG and f(C=0) == ARG and f(dt=7) == ARG
        assert f(eps=-1e-9) == ARG and f(eps=float("nan")) == ARG and f(eps=float("inf")) == ARG
        assert f(R=None) == ARG                       # Hout without a residual
        assert f(C=8193) == UNSUPPORTED
        assert f(X=odd) == ARG and f(R=odd) == ARG and f(H=odd) == ARG and f(w=ctypes.c_void_p(258)) == ARG
        assert f(rows=0) == 0 and f(rows=0, X=None, Y=None) == 0
    assert call(Y=odd) == ARG and call(Y=ctypes.c_void_p(258), dt=F32) == ARG
    assert call8(s=None) == ARG and call8(s=ctypes.c_void_p(258)) == ARG
    q = b._lib.bt_quantize_i8
    assert q(None, 4, 64, BF16, one, one, None) == ARG and q(one, 4, 64, BF16, None, one, None) == ARG
    assert q(one, 4, 64, BF16, one, None, None) == ARG and q(one, 4, 0, BF16, one, one, None) == ARG
    assert q(one, 4, 9000, BF16, one, one, None) == UNSUPPORTED and q(one, 0, 64, BF16, None, None, None) == 0


def test_norm_backward(b):
    size = b.bt_rms_norm_backward_workspace_size
    assert size(-1, 64) == 0 and size(8, 0) == 0 and size(8, 8193) == 0
    assert size(1, 64) >= 256 and size(8, 64) >= 8 * 64 * 4 and size(0, 64) > 0
    assert size(10 ** 9, 64) == size(10 ** 6, 64)     # bounded by the blocks of the launch
    n = size(8, 64)

    def call(dY=one, dH=one, h=one, w=one, rows=8, C=64, eps=1e-6, dt=BF16, dX=one, dw=one, ws=one, nb=n):
        return b._lib.bt_rms_norm_backward(dY, dH, h, w, rows, C, eps, dt, dX, dw, ws, nb, None)
    for k in ("dY", "h", "dX"):
        assert call(**{k: None}) == ARG
    for k in ("dY", "dH", "h", "dX", "dw"):
        assert call(**{k: odd}) == ARG
    assert call(ws=None) == WORKSPACE and call(nb=n - 1) == WORKSPACE and call(ws=ctypes.c_void_p(128)) == ARG
    assert call(eps=-1.0) == ARG and call(dt=3) == ARG and call(C=8193) == UNSUPPORTED
    assert call(rows=0, dw=None, ws=None) == 0


def test_project_i8(b):
    def call(X=one, xs=one, rows=64, C=64, W=one, ws=one, H=2, d=32, dt=BF16, perm=one, inv=one, npad=64, Q=one,
             K=one, V=one):
        return b._lib.bt_qkv_project_i8(X, xs, rows, C, W, ws, H, d, dt, perm, inv, npad, Q, K, V, None)
    for k in ("X", "xs", "W", "ws", "inv", "Q", "K", "V"):
        assert call(**{k: None}) == ARG
    for k in ("xs", "ws", "perm", "inv"):
        assert call(**{k: ctypes.c_void_p(258)}) == ARG
    assert call(Q=odd) == ARG and call(V=ctypes.c_void_p(258), dt=F32) == ARG
    assert call(rows=-1) == ARG and call(C=0) == ARG and call(H=0) == ARG and call(d=0) == ARG and call(dt=2) == ARG
    assert call(npad=-1) == ARG
    assert call(C=65537) == UNSUPPORTED and call(H=700) == UNSUPPORTED and call(rows=2 ** 31) == UNSUPPORTED
    assert call(rows=0, npad=0) == 0 and call(rows=0, perm=None, X=None, Q=None) == 0


def test_layer_i8(b):
    size = b._lib.bt_projected_i8_workspace_size
    n = size(1024, 1000, 64, 8, 32, BF16)
    assert n >= 1000 * 64 + 1000 * 4 + 3 * 1024 * 8 * 32 * 2 + 1000 * 4
    assert size(1024, 1000, 64, 8, 32, F32) > n
    assert size(-1, 10, 64, 8, 32, BF16) == 0 and size(10, 10, 0, 8, 32, BF16) == 0 and size(10, 10, 64, 8, 32, 5) == 0

    def call(X=one, R=one, g=one, eps=1e-6, perm=one, npad=1024, rows=1000, C=64, W=one, ws=one, m=128, H=8, d=32,
             dt=BF16, h=one, O=one, work=one, nb=n):
        return b._lib.bt_projected_ball_attention_i8(X, R, g, eps, perm, npad, rows, C, W, ws, m, H, d, dt, h, O,
                                                     work, nb, None)
    for k in ("X", "W", "ws", "O"):
        assert call(**{k: None}) == ARG
    assert call(O=ctypes.c_void_p(264)) == ARG
    assert call(eps=-1.0) == ARG and call(R=None) == ARG and call(dt=9) == ARG and call(perm=None) == ARG
    assert call(m=0) == SHAPE and call(m=257) == SHAPE and call(d=48) == SHAPE and call(npad=1000) == SHAPE
    assert call(work=None) == WORKSPACE and call(nb=n - 1) == WORKSPACE and call(work=ctypes.c_void_p(272)) == ARG
    assert call(C=8193, nb=1 << 40) == UNSUPPORTED and call(H=700, nb=1 << 40) == UNSUPPORTED
    assert call(rows=0) == 0


def test_layer_i8_of_no_rows(b):
    # an empty batch is served: its workspace has a size, which tells it from a refusal
    assert b._lib.bt_projected_i8_workspace_size(0, 0, 64, 8, 32, BF16) > 0
    assert b._lib.bt_projected_i8_workspace_size(0, 0, 64, 0, 32, BF16) == 0
