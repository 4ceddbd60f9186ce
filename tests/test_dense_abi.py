"""Host-side checks of the dense operators' entry points: bad arguments are
refused before any CUDA call. No call here reaches a launch: each fails one
host-side check, so they are safe with or without a GPU."""
import ctypes

import pytest
import torch

import mxfp4_routed_expert_04_b200 as M

FAKE = 1 << 20          # 16-byte aligned, never dereferenced (validation fails first)
BIG = 1 << 40


def lin(**kw):
    return M.MoeLinearDims(**{**dict(T=4, N=64, K=128), **kw})


def blk(**kw):
    return M.MoeFfnDims(**{**dict(T=4, H=128, I=64, fn=1), **kw})


def error():
    return M._lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,status,text", [
    (dict(T=0), 2, "T="), (dict(T=65537), 2, "T="), (dict(N=4), 2, "N="), (dict(N=100), 2, "N="),
    (dict(K=0), 2, "K="), (dict(K=65544), 2, "K="), (dict(fn=4), 1, "fn"), (dict(fn=-1), 1, "fn"),
    (dict(dtype=2), 1, "dtype"), (dict(out_f32=2), 1, "out_f32"), (dict(ldx=120), 2, "ldx"), (dict(ldx=132), 2, "ldx"),
    (dict(ldy=-8), 2, "ldy"), (dict(ldr=1 << 31), 2, "ldr"),
])
def test_linear_dims_are_refused(kw, status, text):
    d = lin(**kw)
    assert M._lib.moe_linear_workspace_size(ctypes.byref(d)) == 0
    with pytest.raises(M.MoeError):
        M.moe_linear_workspace_size(d)
    st = M._lib.moe_linear(ctypes.byref(d), FAKE, FAKE, None, None, FAKE, None, FAKE, BIG, None)
    assert st == status and text in error()
    st = M._lib.moe_linear_backward(ctypes.byref(d), FAKE, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, BIG, None)
    assert st == status


@pytest.mark.parametrize("kw,status,text", [
    (dict(T=0), 2, "T="), (dict(H=12), 2, "H="), (dict(I=65544), 2, "I="), (dict(fn=9), 1, "fn"),
    (dict(dtype=-1), 1, "dtype"), (dict(save=3), 1, "save"), (dict(reserved=1), 1, "reserved"),
    (dict(ldx=64), 2, "ldx"), (dict(ldy=129), 2, "ldy"), (dict(ldr=8), 2, "ldr"),
])
def test_ffn_dims_are_refused(kw, status, text):
    d = blk(**kw)
    assert M._lib.moe_ffn_workspace_size(ctypes.byref(d)) == 0
    st = M._lib.moe_ffn(ctypes.byref(d), *[FAKE] * 6, None, FAKE, BIG, None)
    assert st == status and text in error()


def test_null_dims():
    assert M._lib.moe_linear(None, FAKE, FAKE, None, None, FAKE, None, FAKE, BIG, None) == 1
    assert M._lib.moe_ffn(None, *[FAKE] * 6, None, FAKE, BIG, None) == 1
    assert M._lib.moe_linear_workspace_size(None) == 0


def test_linear_pointers():
    d = lin()
    n = M.moe_linear_workspace_size(d)

    def call(x=FAKE, w=FAKE, b=None, r=None, y=FAKE, pre=None, ws=FAKE, nws=n, dims=d):
        return M._lib.moe_linear(ctypes.byref(dims), x, w, b, r, y, pre, ws, nws, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None)):
        assert call(**kw) == 1 and "NULL" in error()
    for k in ("x", "w", "b", "r", "y", "pre", "ws"):
        assert call(**{k: FAKE + 2}) == 3, k
    assert call(nws=n - 1) == 4
    # y as its own residual: only with the residual's type and pitch
    assert call(r=FAKE, dims=lin(out_f32=1)) == 1 and "residual" in error()
    assert call(r=FAKE, dims=lin(ldy=72)) == 1


def test_linear_backward_pointers():
    def call(dims, dy=FAKE, x=FAKE, w=FAKE, pre=None, dx=FAKE, dw=FAKE, db=None, ws=FAKE, nws=BIG):
        return M._lib.moe_linear_backward(ctypes.byref(dims), dy, x, w, pre, dx, dw, db, ws, nws, None)

    d, a = lin(), lin(fn=1)
    assert call(d, dy=None) == 1
    assert call(d, dx=None, dw=None) == 1 and "all NULL" in error()
    assert call(d, w=None) == 1 and call(d, x=None) == 1
    assert call(a) == 1 and "pre is NULL" in error()
    assert call(d, pre=FAKE) == 1 and "MOE_FN_NONE" in error()
    for k in ("dy", "x", "w", "dx", "dw", "db"):
        assert call(d, **{k: FAKE + 8}) == 3, k
    assert call(a, pre=FAKE + 8) == 3
    assert call(a, pre=FAKE, nws=M.moe_linear_workspace_size(a) - 1) == 4


def saved(**kw):
    return M._FfnSavedPtrs(**kw)


def test_ffn_saved_buffers():
    def fwd(dims, s):
        return M._lib.moe_ffn(ctypes.byref(dims), FAKE, FAKE, FAKE, FAKE, None, FAKE,
                              ctypes.byref(s) if s is not None else None, FAKE, BIG, None)

    gu = dict(g=FAKE, u=FAKE)
    sc = dict(g_s=FAKE, u_s=FAKE)
    assert fwd(blk(), saved(**gu)) == 1 and "SAVE_NONE" in error()
    assert fwd(blk(save=1), None) == 1
    assert fwd(blk(save=1), saved(g=FAKE)) == 1
    assert fwd(blk(save=1), saved(**gu, **sc)) == 1
    assert fwd(blk(save=2), saved(**gu)) == 1
    assert fwd(blk(save=2), saved(**gu, **sc, x_q=FAKE)) == 1 and "both or neither" in error()
    assert fwd(blk(save=2), saved(g=FAKE, u=FAKE + 4, **sc)) == 3
    assert fwd(blk(save=2), saved(**gu, **sc, x_q=FAKE + 4, x_s=FAKE)) == 3


def test_ffn_backward_pointers():
    def call(dims, s=saved(g=FAKE, u=FAKE), dy=FAKE, x=FAKE, wg=FAKE, wu=FAKE, wd=FAKE, dx=FAKE, dwg=FAKE, dwu=FAKE,
             dwd=FAKE, ws=FAKE, nws=BIG):
        return M._lib.moe_ffn_backward(ctypes.byref(dims), dy, x, wg, wu, wd, ctypes.byref(s) if s else None, dx, dwg,
                                       dwu, dwd, ws, nws, None)

    d = blk(save=1)
    assert call(blk(), None) == 1 and "SAVE_NONE" in error()
    assert call(d, None) == 1
    assert call(d, dy=None) == 1 and call(d, wd=None) == 1
    assert call(d, wg=None) == 1 and call(d, wu=None) == 1
    assert call(d, dwg=None) == 1 and "both or neither" in error()
    assert call(d, dx=None, dwg=None, dwu=None, dwd=None) == 1
    assert call(d, x=None) == 1 and "x_q" in error()
    for k in ("dy", "x", "wg", "wu", "wd", "dx", "dwg", "dwu", "dwd"):
        assert call(d, **{k: FAKE + 4}) == 3, k
    assert call(d, nws=M.moe_ffn_workspace_size(d) - 1) == 4


def test_checkpoint_arguments():
    p, u = M._lib.moe_ckpt8_pack, M._lib.moe_ckpt8_unpack
    assert p(2, 4, 64, FAKE, 0, FAKE, FAKE, None) == 1
    for rows, cols, ld in ((0, 64, 0), (1 << 31, 64, 0), (4, 60, 0), (4, 0, 0), (4, 64, 60), (4, 64, 68)):
        assert p(0, rows, cols, FAKE, ld, FAKE, FAKE, None) == 2
        assert u(0, rows, cols, FAKE, FAKE, FAKE, ld, None) == 2
    assert p(0, 4, 64, None, 0, FAKE, FAKE, None) == 1 and p(0, 4, 64, FAKE, 0, None, FAKE, None) == 1
    assert p(0, 4, 64, FAKE + 2, 0, FAKE, FAKE, None) == 3 and p(0, 4, 64, FAKE, 0, FAKE, FAKE + 1, None) == 3
    assert u(0, 4, 64, FAKE, None, FAKE, 0, None) == 1 and u(0, 4, 64, FAKE, FAKE, FAKE + 2, 0, None) == 3


def test_dense_workspaces():
    assert M._lib.moe_dense_workspace_init(None, 256, None) == 1
    assert M._lib.moe_dense_workspace_init(FAKE, 255, None) == 4
    assert M._lib.moe_dense_workspace_init(FAKE + 8, 256, None) == 3
    # the activation's gradient needs room, its absence none
    assert M.moe_linear_workspace_size(lin(T=1024, fn=1)) >= M.moe_linear_workspace_size(lin(T=1024)) + 1024 * 64 * 2
    sizes = [M.moe_ffn_workspace_size(blk(T=1024, save=s)) for s in (0, 1, 2)]
    assert sizes[0] >= 1024 * 64 * 2 and sizes[1] >= 3 * 1024 * 64 * 2 and sizes[2] >= sizes[1] + 1024 * 128 * 2


def test_binding_checks_tensors():
    """The binding refuses tensors of another type, shape, layout or device."""
    d = lin()
    ok = dict(x=torch.zeros(4, 128, dtype=torch.bfloat16), w=torch.zeros(64, 128, dtype=torch.bfloat16))

    def ptr(t, ld=0, shape=(4, 128)):
        return M._tensor(t, "x", torch.bfloat16, shape, ld, M._device())

    with pytest.raises(M.MoeError, match="float32"):
        ptr(ok["x"].float())
    with pytest.raises(M.MoeError, match="shape"):
        ptr(ok["x"][:3])
    on_dev = ok["x"].get_device()                # the layout checks, as if it were the current device
    with pytest.raises(M.MoeError, match="strides"):
        M._tensor(torch.zeros(128, 4, dtype=torch.bfloat16).t(), "x", torch.bfloat16, (4, 128), 0, on_dev)
    with pytest.raises(M.MoeError, match="strides"):
        M._tensor(ok["x"], "x", torch.bfloat16, (4, 128), 136, on_dev)
    with pytest.raises(M.MoeError, match="not on the current CUDA device"):
        ptr(ok["x"])
    with pytest.raises(M.MoeError, match="workspace"):
        M.moe_linear(d, ok["x"], ok["w"], None, None, ok["x"], None, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(M.MoeError, match="2-D"):
        M.moe_ckpt8_pack(torch.zeros(4, 64), None, None)
    with pytest.raises(M.MoeError, match="x is None"):
        ptr(None)
    with pytest.raises(M.MoeError, match="SAVE_NONE"):
        M.FfnSaved(blk(), device="cpu")
