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


# --- outputs that overlap --------------------------------------------------------------

BASE = 1 << 33          # addresses of buffers that nothing reads: a call that is not refused has no GPU to go to
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass their checks would launch")


class Place:
    """Where every buffer of a call lies: far apart, but for those that `kw` names."""

    def __init__(self, kw):
        self.kw, self.next = kw, BASE

    def __call__(self, name):
        self.next += 1 << 26
        return self.kw.get(name, self.next)


def linear_call(dims, res=False, with_pre=False, **kw):
    p = Place(kw)
    ws = p("ws")
    return M._lib.moe_linear(ctypes.byref(dims), p("x"), p("w"), p("bias"), p("residual") if res else None, p("y"),
                             p("pre") if with_pre else None, ws, BIG, None)


def linear_backward_call(dims, want=("dx", "dw", "dbias"), **kw):
    p = Place(kw)
    return M._lib.moe_linear_backward(
        ctypes.byref(dims), p("dy"), p("x"), p("w"), p("pre") if dims.fn else None,
        *[p(n) if n in want else None for n in ("dx", "dw", "dbias")], p("ws"), BIG, None)


def ffn_saved_at(dims, p):
    n = {0: (), 1: ("g", "u"), 2: ("g", "u", "g_s", "u_s", "x_q", "x_s")}[dims.save]
    return ctypes.byref(saved(**{k: p(k) for k in n})) if n else None


def ffn_call(dims, res=True, **kw):
    p = Place(kw)
    s = ffn_saved_at(dims, p)
    return M._lib.moe_ffn(ctypes.byref(dims), p("x"), p("wg"), p("wu"), p("wd"), p("residual") if res else None, p("y"),
                          s, p("ws"), BIG, None)


def ffn_backward_call(dims, want=("dx", "dwg", "dwu", "dwd"), with_x=True, **kw):
    p = Place(kw)
    s = ffn_saved_at(dims, p)
    return M._lib.moe_ffn_backward(ctypes.byref(dims), p("dy"), p("x") if with_x else None, p("wg"), p("wu"), p("wd"), s,
                                   *[p(n) if n in want else None for n in ("dx", "dwg", "dwu", "dwd")], p("ws"), BIG,
                                   None)


@pytest.mark.parametrize("call,dims,pairs", [
    (linear_call, lin(N=128), ["x y", "w y", "bias y", "ws y", "x ws", "w ws"]),
    (lambda d, **kw: linear_call(d, res=True, with_pre=True, **kw), lin(N=128, fn=1),
     ["x y", "x pre", "y pre", "residual pre", "w pre", "pre ws", "residual ws"]),
    (linear_backward_call, lin(fn=1), ["dy dx", "dy dw", "x dx", "x dw", "w dx", "w dw", "pre dx", "pre dw", "dy dbias",
                                       "pre dbias", "dx dw", "dx dbias", "dw dbias", "dx ws", "dy ws", "pre ws"]),
    (ffn_call, blk(T=64, save=2), ["wg y", "wu y", "wd y", "x g", "x x_q", "x x_s", "x ws", "wd g_s", "g u", "g g_s",
                                   "g_s u_s", "g y", "x_q x_s", "residual u", "residual x_q", "ws y", "ws g", "u x_q"]),
    (ffn_backward_call, blk(save=1), ["dy dx", "dy dwd", "x dx", "x dwg", "wg dx", "wu dwu", "wd dwd", "g dx", "u dwu",
                                      "dx dwg", "dwg dwu", "dwd dx", "ws dx", "ws g", "ws dy"]),
    (lambda d, **kw: ffn_backward_call(d, with_x=False, **kw), blk(T=64, save=2),
     ["x_q dwg", "x_s dx", "g_s dwd", "u_s dx", "ws x_q"]),
])
def test_overlapping_buffers_are_refused(call, dims, pairs):
    """One buffer in two places, and one that begins inside the other."""
    for pair in pairs:
        a, b = pair.split()
        for off in (0, 16):
            assert call(dims, **{a: BASE, b: BASE + off}) == 1 and "overlaps" in error(), (pair, off)
            assert call(dims, **{a: BASE + off, b: BASE}) == 1 and "overlaps" in error(), (pair, off)


def test_in_place_calls_that_are_refused():
    """y = x + f(W x) in place: y is the residual, but also the x that other CTAs still read."""
    assert linear_call(lin(N=128), res=True, x=BASE, residual=BASE, y=BASE) == 1 and "y overlaps x" in error()
    assert linear_call(lin(N=128, ldx=256, ldy=256), x=BASE, y=BASE + 16) == 1
    # a residual shifted against y by a row
    assert linear_call(lin(), res=True, residual=BASE, y=BASE + 128) == 1 and "residual" in error()
    p = M._lib.moe_ckpt8_pack, M._lib.moe_ckpt8_unpack
    far = BASE + (1 << 20)
    assert p[0](0, 4, 64, BASE, 0, BASE, far, None) == 1 and p[0](0, 4, 64, BASE, 0, far, BASE + 496, None) == 1
    assert p[0](0, 4, 64, far, 0, BASE, BASE + 240, None) == 1 and "overlaps" in error()
    assert p[1](0, 4, 64, BASE, far, BASE + 240, 0, None) == 1 and p[1](0, 4, 64, far, BASE, BASE, 0, None) == 1


@NO_GPU
def test_neighbours_are_not_refused():
    """Buffers side by side, or woven into each other's gaps, and what a call does not read."""
    def passes(status):
        return status == 5 or pytest.fail(f"status {status}: {error()}")      # no device: behind all the checks

    # [x | y] and [y | x], column slices of one buffer; x between y's rows with another pitch
    d = lin(N=64, K=64, ldx=128, ldy=128)
    passes(linear_call(d, x=BASE, y=BASE + 128))
    passes(linear_call(d, x=BASE + 128, y=BASE))
    assert linear_call(d, x=BASE, y=BASE + 112) == 1
    assert linear_call(d, x=BASE, y=BASE + 144) == 1
    passes(linear_call(lin(T=2, N=64, K=64, ldx=64, ldy=256), x=BASE + 128, y=BASE))        # 2 rows in a gap
    assert linear_call(lin(T=4, N=64, K=64, ldx=64, ldy=256), x=BASE + 128, y=BASE) == 1    # 4 rows do not fit
    # back to back
    passes(linear_call(lin(), y=BASE, x=BASE + 4 * 64 * 2))
    passes(linear_call(lin(), x=BASE, y=BASE + 4 * 128 * 2))
    # y into its residual; the block's y into x, with x as the residual or not
    passes(linear_call(lin(), res=True, residual=BASE, y=BASE))
    for save in (0, 1, 2):
        passes(ffn_call(blk(save=save), res=False, x=BASE, y=BASE))
        passes(ffn_call(blk(save=save), x=BASE, residual=BASE, y=BASE))
    # gradients over what the call does not read
    passes(linear_backward_call(lin(), want=("dx",), x=BASE, dx=BASE))
    passes(linear_backward_call(lin(), want=("dw",), w=BASE, dw=BASE))
    passes(ffn_backward_call(blk(save=1), want=("dx",), x=BASE, dx=BASE))
    passes(ffn_backward_call(blk(save=1), want=("dwg", "dwu"), wg=BASE, dwg=BASE))
    passes(ffn_backward_call(blk(save=2), x_q=BASE, dx=BASE))         # x is given
    # every buffer that a call can have, each in a place of its own
    passes(linear_call(lin(), res=True, with_pre=True))
    passes(linear_backward_call(lin(fn=1)))
    passes(ffn_call(blk(save=2)))
    passes(ffn_backward_call(blk(save=2)))
    passes(ffn_backward_call(blk(save=2), with_x=False))
    # one input twice
    passes(ffn_call(blk(), wg=BASE, wu=BASE, x=BASE))


@NO_GPU
def test_overlap_is_exact():
    """Pitched rows against pitched rows, byte by byte."""
    import random
    rng = random.Random(5)
    seen = set()
    for _ in range(3000):
        T, N, K = rng.randint(1, 5), 8 * rng.randint(1, 6), 8 * rng.randint(1, 6)
        ldx = K + 8 * rng.randint(0, 14)
        ldy = ldx if rng.random() < 0.4 and ldx >= N else N + 8 * rng.randint(0, 14)
        off = 16 * rng.randint(-60, 60)
        xs = {2 * (t * ldx + k) // 16 for t in range(T) for k in range(K)}
        ys = {(off + 2 * (t * ldy + k)) // 16 for t in range(T) for k in range(N)}
        want = 1 if xs & ys else 5
        seen.add((want, ldx == ldy))
        assert linear_call(lin(T=T, N=N, K=K, ldx=ldx, ldy=ldy), x=BASE, y=BASE + off) == want, (T, N, K, ldx, ldy, off)
    assert len(seen) == 4
