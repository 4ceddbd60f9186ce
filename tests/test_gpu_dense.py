"""The dense operators on the GPU against plain fp64 forms: the projection with
a fused epilogue, the gated feed-forward block, their backward passes and the
8-bit activation checkpoints. Bounds: dense_reference."""
import pytest
import torch

import dense_reference as R
import mxfp4_routed_expert_04_b200 as M

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def code(dt):
    return M.DTYPE_F16 if dt is HF else M.DTYPE_BF16


def rand(shape, std, dt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def empty(shape, dt):
    """An output buffer of NaN: whatever is not written shows."""
    return torch.full(shape, float("nan"), dtype=dt, device="cuda")


def workspace(size):
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    M.moe_dense_workspace_init(ws)
    return ws


def pitched(t, ld, fill=float("nan")):
    """A copy of t whose rows lie ld elements apart, the gaps filled; (view, whole buffer)."""
    buf = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]], buf


# --- projection --------------------------------------------------------------------

LINEAR = [
    # T, N, K, type, fn, bias, residual, fp32 out
    (1, 8, 8, BF, "none", False, False, False),
    (1, 2048, 1024, BF, "none", True, True, False),
    (1, 136, 1000, HF, "silu", True, False, False),
    (2, 264, 72, BF, "gelu", True, True, False),
    (3, 4096, 264, HF, "none", False, True, False),
    (7, 520, 4104, BF, "relu", True, False, True),
    (16, 1024, 2048, BF, "none", False, True, False),
    (17, 72, 8200, HF, "none", True, False, True),
    (31, 1000, 512, BF, "silu", False, False, False),
    (33, 256, 256, HF, "gelu", True, True, False),
    (63, 640, 1288, BF, "none", True, True, True),
    (64, 2056, 776, BF, "none", False, False, False),
    (65, 72, 64, HF, "relu", True, True, False),
    (100, 384, 4096, BF, "none", True, True, False),
    (128, 128, 128, BF, "none", False, False, False),
    (129, 264, 136, HF, "silu", True, True, False),
    (255, 200, 1000, BF, "none", True, False, False),
    (257, 520, 520, BF, "gelu", False, True, True),
    (333, 1000, 776, HF, "gelu", True, False, False),
    (700, 2312, 136, BF, "none", True, True, False),
    (1031, 1288, 328, HF, "none", False, True, False),
    # few and long tiles: K divided over clusters
    (66, 264, 4096, BF, "none", True, True, False),
    (100, 1024, 8192, BF, "silu", True, False, False),
    (129, 520, 5000, HF, "gelu", True, True, True),
    (300, 200, 4104, BF, "none", False, True, False),
    (1000, 512, 2048, BF, "relu", True, True, False),
    # several tiles a CTA
    (2100, 5008, 328, HF, "silu", True, True, False),
    (1500, 3336, 1096, BF, "none", False, True, True),
    (130, 21000, 72, BF, "none", True, False, False),
]


@pytest.mark.parametrize("T,N,K,dt,fn,bias,res,f32", LINEAR)
def test_linear(T, N, K, dt, fn, bias, res, f32):
    x, w = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2)
    b = rand((N,), 0.5, dt, 3) if bias else None
    r = rand((T, N), 1, dt, 4) if res else None
    out = F32 if f32 else dt
    d = M.MoeLinearDims(T=T, N=N, K=K, fn=R.FN[fn], dtype=code(dt), out_f32=int(f32))
    ws = workspace(M.moe_linear_workspace_size(d))
    y, pre = empty((T, N), out), empty((T, N), dt)
    M.moe_linear(d, x, w, b, r, y, pre, ws)
    ref, rpre = R.linear(x, w, b, r, fn, dt, out)
    R.check(y, ref, "y", None if f32 else 1, dt)
    R.check(pre, rpre, "pre", 1, dt)
    y2 = empty((T, N), out)
    M.moe_linear(d, x, w, b, r, y2, None, ws)
    assert torch.equal(y, y2), "the same inputs gave other bits"
    assert M.moe_device_status(ws) == 0


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_linear_on_pitched_rows(T):
    """Rows further apart than they are long, NaN between them, y and residual of other pitches."""
    N, K, dt = 264, 200, BF
    x, w, r = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2), rand((T, N), 1, dt, 4)
    xv, _ = pitched(x, 256)
    rv, _ = pitched(r, 272)
    _, ybuf = pitched(torch.zeros(T + 3, N, dtype=dt), 320, 7.0)
    ybuf[T:] = 7.0
    yv = ybuf[:T, :N]
    d = M.MoeLinearDims(T=T, N=N, K=K, ldx=256, ldy=320, ldr=272)
    M.moe_linear(d, xv, w, None, rv, yv, None, workspace(M.moe_linear_workspace_size(d)))
    R.check(yv, R.linear(x, w, None, r, "none", dt, dt)[0], "y", 1, dt)
    assert (ybuf[:, N:] == 7.0).all(), "elements between the rows were written"
    assert (ybuf[T:] == 7.0).all(), "rows behind the last were written"


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_into_its_residual(T):
    N, K, dt = 520, 136, BF
    x, w, r = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2), rand((T, N), 1, dt, 4)
    ref = R.linear(x, w, None, r, "none", dt, dt)[0]
    d = M.MoeLinearDims(T=T, N=N, K=K)
    M.moe_linear(d, x, w, None, r, r, None, workspace(M.moe_linear_workspace_size(d)))
    R.check(r, ref, "y", 1, dt)


@pytest.mark.parametrize("T", [1, 3, 50, 300])
def test_non_finite_inputs_stay_in_their_rows_and_columns(T):
    N, K, dt = 264, 136, BF
    x, w = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2)
    ref = R.linear(x, w, None, None, "none", dt, dt)[0]
    x, w = x.clone(), w.clone()
    x[T - 1, 5] = float("nan")
    w[N - 1, 7] = float("inf")
    d = M.MoeLinearDims(T=T, N=N, K=K)
    y = empty((T, N), dt)
    M.moe_linear(d, x, w, None, None, y, None, workspace(M.moe_linear_workspace_size(d)))
    assert y[T - 1].isnan().all()
    if T > 1:
        assert y[:-1, N - 1].isinf().all()
        R.check(y[:-1, :N - 1], (ref[0][:-1, :N - 1], ref[1][:-1, :N - 1]), "y", 1, dt)


def test_linear_offsets_past_32_bits():
    """65536 x 65536 outputs: element offsets past 2^32."""
    T = N = 65536
    K, dt = 16, BF
    x, w = rand((T, K), 1, dt, 1), rand((N, K), 0.3, dt, 2)
    d = M.MoeLinearDims(T=T, N=N, K=K)
    y = empty((T, N), dt)
    M.moe_linear(d, x, w, None, None, y, None, workspace(M.moe_linear_workspace_size(d)))
    for r0 in (0, 32760, 65500):
        rows = slice(r0, r0 + 36)
        R.check(y[rows], R.linear(x[rows], w, None, None, "none", dt, dt)[0], "y", 1, dt)
    assert not y[::97].isnan().any()


LINEAR_GRAD = [
    (1, 8, 8, BF, "none", False, False),
    (1, 264, 136, HF, "silu", True, False),
    (5, 136, 1000, BF, "gelu", True, True),
    (16, 520, 256, BF, "none", True, False),
    (33, 72, 520, HF, "relu", False, False),
    (64, 256, 256, BF, "silu", True, False),
    (130, 264, 392, HF, "none", True, True),
    (300, 1000, 520, BF, "gelu", True, False),
    (777, 328, 1352, HF, "silu", False, False),
    # few tokens against large weights; T above the few with long sums
    (2, 2056, 1000, BF, "silu", True, False),
    (9, 1000, 776, HF, "none", True, True),
    (50, 1288, 520, HF, "gelu", True, False),
    (70, 4104, 264, BF, "relu", True, False),
    (2000, 2056, 3000, BF, "none", False, False),
    (4100, 1288, 1352, HF, "gelu", True, False),
]


@pytest.mark.parametrize("T,N,K,dt,fn,bias,f32", LINEAR_GRAD)
def test_linear_backward(T, N, K, dt, fn, bias, f32):
    x, w, dy = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2), rand((T, N), 0.3, dt, 3)
    pre = rand((T, N), 1.5, dt, 4) if fn != "none" else None
    out = F32 if f32 else dt
    d = M.MoeLinearDims(T=T, N=N, K=K, fn=R.FN[fn], dtype=code(dt), out_f32=int(f32))
    ws = workspace(M.moe_linear_workspace_size(d))
    got = {"dx": empty((T, K), out), "dw": empty((N, K), out), "db": empty((N,), out) if bias else None}
    M.moe_linear_backward(d, dy, x, w, pre, got["dx"], got["dw"], got["db"], ws)
    ref = R.linear_grads(dy, x, w, pre, fn, bias, dt, out)
    for n, r in ref.items():
        R.check(got[n], r, n, None if f32 else 2, dt)
    # each alone, without what it does not read
    for n in ref:
        one = {m: torch.full_like(got[m], float("nan")) if m == n else None for m in ("dx", "dw", "db")}
        M.moe_linear_backward(d, dy, x if n == "dw" else None, w if n == "dx" else None, pre, one["dx"], one["dw"],
                              one["db"], ws)
        assert torch.equal(one[n], got[n]), n
    assert M.moe_device_status(ws) == 0


def test_linear_backward_on_pitched_rows():
    T, N, K, dt = 50, 136, 264, BF
    x, w, dy = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2), rand((T, N), 0.3, dt, 3)
    pre = rand((T, N), 1.5, dt, 4)
    d = M.MoeLinearDims(T=T, N=N, K=K, fn=1, ldx=272, ldy=144)
    xv, _ = pitched(x, 272)
    dyv, _ = pitched(dy, 144)
    dxv, dxbuf = pitched(torch.zeros_like(x), 272, 7.0)
    dw, db = empty((N, K), dt), empty((N,), dt)
    M.moe_linear_backward(d, dyv, xv, w, pre, dxv, dw, db, workspace(M.moe_linear_workspace_size(d)))
    ref = R.linear_grads(dy, x, w, pre, "silu", True, dt, dt)
    for n, got in (("dx", dxv), ("dw", dw), ("db", db)):
        R.check(got, ref[n], n, 2, dt)
    assert (dxbuf[:, K:] == 7.0).all()


# --- gated block --------------------------------------------------------------------

FFN = [
    # T, H, I, type, fn, residual, fp32 out
    (1, 8, 8, BF, "silu", False, False),
    (1, 1024, 512, BF, "silu", True, False),
    (1, 1000, 136, HF, "gelu", True, True),
    (2, 264, 1352, BF, "relu", True, False),
    (9, 520, 40, HF, "silu", False, False),
    (16, 1024, 1024, BF, "silu", True, False),
    (32, 2048, 256, BF, "none", True, False),
    (40, 136, 328, HF, "gelu", True, False),
    (65, 264, 520, BF, "silu", True, True),
    (130, 1000, 200, BF, "gelu", False, False),
    (300, 392, 712, HF, "silu", True, False),
    (520, 256, 384, BF, "relu", True, False),
    # long sums: K divided over clusters, or (8-bit checkpoints) in pieces
    (70, 4096, 264, BF, "silu", True, False),
    (200, 2504, 328, HF, "gelu", False, False),
    (1100, 2248, 1544, BF, "silu", True, False),
    (1100, 2248, 2600, HF, "gelu", True, False),
    (2500, 520, 4104, BF, "relu", False, False),
]


def ffn_tensors(T, H, I, dt):
    return (rand((T, H), 1, dt, 1), rand((I, H), 0.05, dt, 2), rand((I, H), 0.05, dt, 3), rand((H, I), 0.05, dt, 4))


@pytest.mark.parametrize("save", [M.SAVE_NONE, M.SAVE_16, M.SAVE_8])
@pytest.mark.parametrize("T,H,I,dt,fn,res,f32", FFN)
def test_ffn(T, H, I, dt, fn, res, f32, save):
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    r = rand((T, H), 1, dt, 5) if res else None
    out = F32 if f32 else dt
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=R.FN[fn], dtype=code(dt), save=save, out_f32=int(f32))
    ws = workspace(M.moe_ffn_workspace_size(d))
    y = empty((T, H), out)
    saved = M.FfnSaved(d) if save else None
    M.moe_ffn(d, x, wg, wu, wd, r, y, saved, ws)
    ref, g, u = R.ffn(x, wg, wu, wd, r, fn, dt, out)
    R.check(y, ref, "y", None if f32 else 2, dt)
    if save == M.SAVE_16:
        R.check(saved.g, (g[0], R.stored(*g, dt)), "g", 1, dt)
        R.check(saved.u, (u[0], R.stored(*u, dt)), "u", 1, dt)
    if save == M.SAVE_8:
        for n, (v, e), q, s in (("g", g, saved.g, saved.g_s), ("u", u, saved.u, saved.u_s)):
            got = R.unpack8(q, s)
            sc = torch.exp2(s.double() - 127).repeat_interleave(32, dim=1)[:, :I]
            # half a step of E4M3: 2^-4 of the value, or of its smallest normal 2^-6
            R.check(got, (v, e + 2.0 ** -4 * (v.abs() + e) + 2.0 ** -10 * sc), n)
            a = torch.nn.functional.pad(v.abs(), (0, -I % 32)).reshape(T, -1, 32).amax(-1)
            top = 448 * torch.exp2(s.double() - 127)
            slack = 1 + 2.0 ** -12
            assert (a <= top * slack).all() and ((a * slack >= top / 2) | (s == 0)).all(), f"{n}: scale"
        check_packed(x, saved.x_q, saved.x_s)
    assert M.moe_device_status(ws) == 0


@pytest.mark.parametrize("T", [1, 6, 70, 300])
def test_ffn_on_pitched_rows_into_its_residual(T):
    H, I, dt = 264, 136, BF
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    r = rand((T, H), 1, dt, 5)
    ref = R.ffn(x, wg, wu, wd, r, "silu", dt, dt)[0]
    xv, _ = pitched(x, 320)
    rv, rbuf = pitched(r, 280, 7.0)
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, ldx=320, ldy=280, ldr=280)
    M.moe_ffn(d, xv, wg, wu, wd, rv, rv, None, workspace(M.moe_ffn_workspace_size(d)))
    R.check(rv, ref, "y", 2, dt)
    assert (rbuf[:, H:] == 7.0).all()


def ffn_buffers(T, H, I, out):
    return {"dx": empty((T, H), out), "dwg": empty((I, H), out), "dwu": empty((I, H), out), "dwd": empty((H, I), out)}


@pytest.mark.parametrize("T,H,I,dt,fn,res,f32", FFN)
def test_ffn_backward(T, H, I, dt, fn, res, f32):
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    dy, out = rand((T, H), 0.3, dt, 6), F32 if f32 else dt
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=R.FN[fn], dtype=code(dt), save=M.SAVE_16, out_f32=int(f32))
    ws = workspace(M.moe_ffn_workspace_size(d))
    saved = M.FfnSaved(d, g=rand((T, I), 1.5, dt, 7), u=rand((T, I), 1.5, dt, 8))
    got = ffn_buffers(T, H, I, out)
    M.moe_ffn_backward(d, dy, x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws)
    ref = R.ffn_grads(dy, x, wg, wu, wd, saved.g, saved.u, fn, dt, out)
    for n, r in ref.items():
        R.check(got[n], r, n, None if f32 else 2, dt)
    # in parts: dx alone, the gate/up pair alone, dwd alone
    for part in (("dx",), ("dwg", "dwu"), ("dwd",)):
        one = {n: torch.full_like(got[n], float("nan")) if n in part else None for n in got}
        M.moe_ffn_backward(d, dy, x if "dwg" in part else None, wg if "dx" in part else None,
                           wu if "dx" in part else None, wd, saved, one["dx"], one["dwg"], one["dwu"], one["dwd"], ws)
        for n in part:
            assert torch.equal(one[n], got[n]), n
    assert M.moe_device_status(ws) == 0


@pytest.mark.parametrize("keep_x", [True, False])
@pytest.mark.parametrize("T,H,I,dt,fn,res,f32", FFN)
def test_ffn_backward_from_8_bits(T, H, I, dt, fn, res, f32, keep_x):
    """Forward with 8-bit checkpoints, then the gradients of what they hold."""
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    dy, out = rand((T, H), 0.3, dt, 6), F32 if f32 else dt
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=R.FN[fn], dtype=code(dt), save=M.SAVE_8, out_f32=int(f32))
    ws = workspace(M.moe_ffn_workspace_size(d))
    saved, y, got = M.FfnSaved(d, keep_x=keep_x), empty((T, H), out), ffn_buffers(T, H, I, out)
    M.moe_ffn(d, x, wg, wu, wd, None, y, saved, ws)
    M.moe_ffn_backward(d, dy, None if keep_x else x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"],
                       got["dwd"], ws)
    xs = R.unpack8(saved.x_q, saved.x_s).to(dt) if keep_x else x
    ref = R.ffn_grads(dy, xs, wg, wu, wd, R.unpack8(saved.g, saved.g_s), R.unpack8(saved.u, saved.u_s), fn, dt, out)
    for n, r in ref.items():
        R.check(got[n], r, n, None if f32 else 2, dt)


def test_ffn_gradients_against_differences():
    """Central differences of the fp64 block along random directions."""
    T, H, I, dt = 40, 136, 200, HF
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    dy = rand((T, H), 0.3, dt, 6)
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, dtype=code(dt), save=M.SAVE_16, out_f32=1)
    ws = workspace(M.moe_ffn_workspace_size(d))
    saved, y, got = M.FfnSaved(d), empty((T, H), F32), ffn_buffers(T, H, I, F32)
    M.moe_ffn(d, x, wg, wu, wd, None, y, saved, ws)
    M.moe_ffn_backward(d, dy, x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws)

    def loss(x, wg, wu, wd):
        return (dy.double() * ((R.value("silu", x @ wg.t()) * (x @ wu.t())) @ wd.t())).sum()

    at = [t.double() for t in (x, wg, wu, wd)]
    for i, n in enumerate(("dx", "dwg", "dwu", "dwd")):
        v = rand(at[i].shape, 1, F32, 20 + i).double()
        step = 1e-5
        hi, lo = ([t + s * step * v if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        # g, u, dg, du, h each rounded to f16: at most 5 u of the gradient's size in
        # the direction's, differences in fp64 off by far less
        tol = 5 * R.unit(dt) * got[n].double().norm() * v.norm()
        assert (diff - (got[n].double() * v).sum()).abs() <= tol, n


def test_linear_gradients_against_differences():
    T, N, K, dt = 40, 136, 200, HF
    x, w, b, dy = rand((T, K), 1, dt, 1), rand((N, K), 0.1, dt, 2), rand((N,), 0.5, dt, 3), rand((T, N), 0.3, dt, 4)
    d = M.MoeLinearDims(T=T, N=N, K=K, fn=2, dtype=code(dt), out_f32=1)
    ws = workspace(M.moe_linear_workspace_size(d))
    y, pre = empty((T, N), F32), empty((T, N), dt)
    dx, dw, db = empty((T, K), F32), empty((N, K), F32), empty((N,), F32)
    M.moe_linear(d, x, w, b, None, y, pre, ws)
    M.moe_linear_backward(d, dy, x, w, pre, dx, dw, db, ws)

    def loss(x, w, b):
        return (dy.double() * R.value("gelu", x @ w.t() + b)).sum()

    at = [t.double() for t in (x, w, b)]
    for i, got in enumerate((dx, dw, db)):
        v = rand(at[i].shape, 1, F32, 20 + i).double()
        step = 1e-5
        hi, lo = ([t + s * step * v if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        tol = 5 * R.unit(dt) * got.double().norm() * v.norm()     # pre and dz rounded to f16
        assert (diff - (got.double() * v).sum()).abs() <= tol, i


# --- 8-bit checkpoints ------------------------------------------------------------------

def check_packed(x, q, s):
    qr, sr = R.pack8(x.double().cpu())
    assert torch.equal(s.cpu(), sr), "scales"
    finite = (s.cpu() != 255).repeat_interleave(32, dim=1)[:, :q.shape[1]]
    assert torch.equal(q.cpu()[finite], qr[finite]), "codes"


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 32), (3, 40), (17, 264), (5, 1000), (64, 512)])
def test_ckpt8_round_trip(rows, cols, dt):
    x = (rand((rows, cols), 1, F32, 1) * torch.exp(2 * rand((rows, 1), 1, F32, 2))).to(dt)
    q = torch.zeros((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.zeros((rows, (cols + 31) // 32), dtype=torch.uint8, device="cuda")
    M.moe_ckpt8_pack(x, q, s)
    check_packed(x, q, s)
    back = empty((rows, cols), dt)
    M.moe_ckpt8_unpack(q, s, back)
    assert torch.equal(back, R.unpack8(q, s).to(dt))


def test_ckpt8_special_values():
    big, tiny = torch.finfo(BF).max, 2.0 ** -133
    rows = [
        [0.0] * 32, [-0.0] * 32, [big] * 32, [tiny] * 32, [tiny * k for k in range(32)],
        [448.0] + [0.0] * 31, [449.0 + 1] + [1.0] * 31, [-448.0] + [2.0 ** -9] * 31,
        [448.0] + [17.0 + 2 * k for k in range(31)],          # ties between neighbours 16, 18, 20, ...
        [448.0] + [2.0 ** -10 * k for k in range(31)],        # ties among the subnormals
        [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [float("-inf"), float("nan")] + [0.0] * 30,
        [1.75] + [0.1] * 31, [1.7578125] + [0.1] * 31,
    ]
    x = torch.tensor(rows, dtype=torch.float64).to(BF).cuda()
    q = torch.zeros_like(x, dtype=torch.uint8)
    s = torch.zeros((len(rows), 1), dtype=torch.uint8, device="cuda")
    M.moe_ckpt8_pack(x, q, s)
    check_packed(x, q, s)
    back = empty(tuple(x.shape), BF)
    M.moe_ckpt8_unpack(q, s, back)
    want = R.unpack8(q, s).to(BF)
    assert torch.equal(back.isnan(), want.isnan())
    assert torch.equal(back[~back.isnan()], want[~want.isnan()])
    assert back[10].isnan().all() and back[11].isnan().all() and back[12].isnan().all()
    assert torch.signbit(back[1]).all() and not torch.signbit(back[0]).any()


def test_ckpt8_on_pitched_rows():
    rows, cols = 9, 72
    x = rand((rows, cols), 1, BF, 1)
    xv, _ = pitched(x, 96)
    q = torch.zeros((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.zeros((rows, 3), dtype=torch.uint8, device="cuda")
    M.moe_ckpt8_pack(xv, q, s)
    check_packed(x, q, s)
    bv, buf = pitched(torch.zeros_like(x), 88, 7.0)
    M.moe_ckpt8_unpack(q, s, bv)
    assert torch.equal(bv, R.unpack8(q, s).to(BF)) and (buf[:, cols:] == 7.0).all()


def test_ckpt8_offsets_past_32_bits():
    rows, cols = 66000, 65536
    x = torch.empty((rows, cols), dtype=BF, device="cuda")
    x[:4] = rand((4, cols), 1, BF, 1)
    x[4:-4] = 0
    x[-4:] = rand((4, cols), 1, BF, 2)
    q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda")
    M.moe_ckpt8_pack(x, q, s)
    M.moe_ckpt8_unpack(q, s, x)
    for i, seed in ((slice(0, 4), 1), (slice(-4, None), 2)):
        assert torch.equal(x[i], R.unpack8(q[i], s[i]).to(BF))
        assert ((x[i].double() - rand((4, cols), 1, BF, seed).double()).abs()
                <= 2.0 ** -4 * rand((4, cols), 1, BF, seed).double().abs() + 2.0 ** -10).all()
    assert (x[4:-4:997] == 0).all()


# --- use -------------------------------------------------------------------------------

@pytest.mark.parametrize("T", [1, 24, 300])
def test_captured_calls_follow_their_inputs(T):
    """Two graphs that share a workspace, replayed one after the other on new inputs."""
    H, I, dt = 264, 520, BF
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    wl = rand((I, H), 0.05, dt, 9)
    df = M.MoeFfnDims(T=T, H=H, I=I, fn=1, dtype=code(dt), save=M.SAVE_8)
    dl = M.MoeLinearDims(T=T, N=I, K=H, fn=2, dtype=code(dt))
    ws = workspace(max(M.moe_ffn_workspace_size(df), M.moe_linear_workspace_size(dl)))
    saved, y, z, dy = M.FfnSaved(df), empty((T, H), dt), empty((T, I), dt), rand((T, H), 0.3, dt, 6)
    got = ffn_buffers(T, H, I, dt)

    def block():
        M.moe_ffn(df, x, wg, wu, wd, None, y, saved, ws)
        M.moe_ffn_backward(df, dy, None, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws)

    def lin():
        M.moe_linear(dl, x, wl, None, None, z, None, ws)

    block(), lin()
    torch.cuda.synchronize()
    graphs = []
    for f in (block, lin):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for seed in (31, 32):
        x.copy_(rand((T, H), 1, dt, seed))
        dy.copy_(rand((T, H), 0.3, dt, seed + 10))
        for t in (y, z, *got.values()):
            t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in (y, z, *got.values())]
        block(), lin()
        for a, b in zip(have, (y, z, *got.values())):
            assert torch.equal(a, b)
    del graphs
    R.check(z, R.linear(x, wl, None, None, "gelu", dt, dt)[0], "z", 1, dt)
    R.check(y, R.ffn(x, wg, wu, wd, None, "silu", dt, dt)[0], "y", 2, dt)


def test_calls_on_a_stream_of_their_own():
    T, H, I, dt = 70, 264, 520, BF
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws, y = workspace(M.moe_ffn_workspace_size(d)), empty((T, H), dt)
    s.wait_stream(torch.cuda.current_stream())
    M.moe_ffn(d, x, wg, wu, wd, None, y, None, ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    R.check(y, R.ffn(x, wg, wu, wd, None, "silu", dt, dt)[0], "y", 2, dt)


def test_calls_on_two_streams_at_once():
    """Separate workspaces and outputs, the same inputs: the results of one call at a time."""
    H, I, dt = 520, 1032, BF
    for T in (1, 30, 100, 400):
        x, wg, wu, wd = ffn_tensors(T, H, I, dt)
        d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, save=M.SAVE_8)
        runs = []
        for _ in range(2):
            saved, got = M.FfnSaved(d), ffn_buffers(T, H, I, dt)
            runs.append((torch.cuda.Stream(), workspace(M.moe_ffn_workspace_size(d)), saved, empty((T, H), dt), got))
        torch.cuda.synchronize()
        for _ in range(4):
            for s, ws, saved, y, got in runs:
                M.moe_ffn(d, x, wg, wu, wd, None, y, saved, ws, stream=s)
                M.moe_ffn_backward(d, y, None, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws,
                                   stream=s)
        torch.cuda.synchronize()
        R.check(runs[0][3], R.ffn(x, wg, wu, wd, None, "silu", dt, dt)[0], "y", 2, dt)
        assert torch.equal(runs[0][3], runs[1][3])
        for n in runs[0][4]:
            assert torch.equal(runs[0][4][n], runs[1][4][n]), n


def test_one_output_feeds_the_next_call_as_its_weight():
    """Back to back on one stream, the second reading the first's output as weights."""
    dt = BF
    for T in (3, 40, 90, 200):
        a, b, x = rand((256, 128), 0.3, dt, 1), rand((264, 128), 0.3, dt, 2), rand((T, 264), 1, dt, 3)
        w, y = empty((256, 264), dt), empty((T, 256), dt)
        d1, d2 = M.MoeLinearDims(T=256, N=264, K=128), M.MoeLinearDims(T=T, N=256, K=264)
        ws = workspace(max(M.moe_linear_workspace_size(d1), M.moe_linear_workspace_size(d2)))
        for _ in range(5):
            w.fill_(float("nan"))
            M.moe_linear(d1, a, b, None, None, w, None, ws)
            M.moe_linear(d2, x, w, None, None, y, None, ws)
            R.check(y, R.linear(x, w, None, None, "none", dt, dt)[0], "y", 1, dt)


@pytest.mark.parametrize("save", [M.SAVE_16, M.SAVE_8])
def test_a_training_step_of_a_stack(save):
    """Projection -> gated block with a residual -> projection, forward and
    backward, against the same stack in fp64 with autograd on exact values."""
    T, H, I, dt = 96, 256, 512, HF
    x, wi, bi = rand((T, 128), 1, dt, 1), rand((H, 128), 0.1, dt, 2), rand((H,), 0.3, dt, 3)
    _, wg, wu, wd = ffn_tensors(T, H, I, dt)
    wo, dy = rand((64, H), 0.1, dt, 10), rand((T, 64), 0.3, dt, 11)
    di = M.MoeLinearDims(T=T, N=H, K=128, fn=R.FN["gelu"], dtype=code(dt))
    do = M.MoeLinearDims(T=T, N=64, K=H, dtype=code(dt))
    df = M.MoeFfnDims(T=T, H=H, I=I, fn=1, dtype=code(dt), save=save)
    block = M.MoeFfn(df, {"wg": wg, "wu": wu, "wd": wd})
    wsl = workspace(max(M.moe_linear_workspace_size(di), M.moe_linear_workspace_size(do)))
    a, pre, y = empty((T, H), dt), empty((T, H), dt), empty((T, 64), dt)
    M.moe_linear(di, x, wi, bi, None, a, pre, wsl)
    b = block(a, a)
    M.moe_linear(do, b, wo, None, None, y, None, wsl)
    db, dwo = empty((T, H), dt), empty((64, H), dt)
    M.moe_linear_backward(do, dy, b, wo, None, db, dwo, None, wsl)
    da, dw = block.backward(db, a if save == M.SAVE_16 else None)
    da = da + db                                    # the residual's gradient
    dx, dwi, dbi = empty((T, 128), dt), empty((H, 128), dt), empty((H,), dt)
    M.moe_linear_backward(di, da, x, wi, pre, dx, dwi, dbi, wsl)

    leaves = [t.double().requires_grad_() for t in (x, wi, bi, wg, wu, wd, wo)]
    X, WI, BI, WG, WU, WD, WO = leaves
    A = torch.nn.functional.gelu(X @ WI.t() + BI)
    B = A + (torch.nn.functional.silu(A @ WG.t()) * (A @ WU.t())) @ WD.t()
    Y = B @ WO.t()
    Y.backward(dy.double())
    # relative size of the error: about ten 16-bit roundings on the longest way
    # (10 u); 8-bit checkpoints: x, g and u each off by up to 2^-4, a third of
    # that in the root mean square, entering products of independent errors
    tol = 10 * R.unit(dt) + (3 * 2.0 ** -4 / 3 if save == M.SAVE_8 else 0)
    for n, got, ref in [("y", y, Y.detach())] + [(n, g, t.grad) for n, g, t in zip(
            ("dx", "dwi", "dbi", "dwg", "dwu", "dwd", "dwo"), (dx, dwi, dbi, dw["wg"], dw["wu"], dw["wd"], dwo), leaves)]:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert rel <= tol, f"{n}: {rel:.3e} above {tol:.3e}"


# --- sums in front of a checkpoint --------------------------------------------------------

LONG_H, LONG_I = 65536, 9536


@pytest.fixture(scope="module")
def long_sums():
    """Positive x and weights of the longest contraction, and the exact g and u."""
    x = rand((130, LONG_H), 1, BF, 1).abs()
    w = [rand((LONG_I, LONG_H), 2e-3, BF, 2 + i).abs() for i in range(2)]
    exact = [torch.cat([x.double() @ c.double().t() for c in m.split(1192)], dim=1) for m in w]
    yield x, w, exact
    del x, w, exact
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,I", [(1, LONG_I), (8, LONG_I), (9, LONG_I), (40, LONG_I), (64, LONG_I), (65, LONG_I),
                                 (130, LONG_I), (8, 4104), (40, 4104), (3, 72), (64, 72), (130, 72)])
def test_codes_of_long_sums(long_sums, T, I):
    """The 8-bit g and u of K = 65536. All products are positive, so no partial
    sum is above the whole, S. In pieces of K = 1024 a tensor-core sum has 64
    additions, each off by at most 2^-23 of its piece: the pieces together by
    64 * 2^-23 S; adding up 64 pieces and the parts of up to 8 CTAs rounds 72
    times by 2^-24 S. In one piece of all K, 4096 additions cut
    off, one code in 100 is another."""
    x, w, exact = long_sums
    d = M.MoeFfnDims(T=T, H=LONG_H, I=I, fn=1, save=M.SAVE_8)
    saved, y = M.FfnSaved(d, keep_x=False), empty((T, LONG_H), BF)
    wd = torch.zeros((LONG_H, I), dtype=BF, device="cuda")
    ws = workspace(M.moe_ffn_workspace_size(d))
    M.moe_ffn(d, x[:T], w[0][:I], w[1][:I], wd, None, y, saved, ws)
    rel = 64 * 2.0 ** -23 + 72 * 2.0 ** -24
    for n, v, q, s in (("g", exact[0], saved.g, saved.g_s), ("u", exact[1], saved.u, saved.u_s)):
        assert R.check_codes(v[:T, :I], rel, q, s, n) > 0.99 * T * I
    assert (y == 0).all() and M.moe_device_status(ws) == 0


# --- activations over their whole range --------------------------------------------------

def arguments(dt):
    """512 arguments of an activation: a grid over [-13, 13], ever larger ones, both zeros."""
    z = torch.linspace(-13, 13, 470, dtype=torch.float64)
    far = torch.tensor([0.0, 1e-7, 14.0, 17.0, 20.0, 40.0, 60.0, 80.0, 86.0, 87.0, 87.5, 88.0, 88.5, 89.0, 104.0, 300.0,
                        1e3, 1e4, 3e4, 6e4, torch.finfo(dt).max], dtype=torch.float64)
    return torch.cat([z, far, -far]).to(dt)


def exp_unit(a):
    """Relative bound of __expf at a, as the CUDA programming guide states it, and of a's own rounding."""
    return (2 + 1.173 * a.abs()) * 2.0 ** -23 + a.abs() * 2.0 ** -24


@pytest.mark.parametrize("T", [1, 16, 80])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("fn", ["silu", "gelu", "relu"])
def test_activation_values_over_their_range(fn, dt, T):
    """In fp32, through a projection by the identity (its sums are exact).
    silu: the exponential, 1 + e, the quotient (2 units; 0 once the divisor
    passes 2^126) and a last rounding. gelu: the exponential, a quotient, the
    fitted polynomial (5.5e-7) and three products of the tail; above 0 the
    complement rounds once more."""
    z = arguments(dt)[:512].cuda()
    n = z.numel()
    x = z.expand(T, n).contiguous()
    d = M.MoeLinearDims(T=T, N=n, K=n, fn=R.FN[fn], dtype=code(dt), out_f32=1)
    y = empty((T, n), F32)
    M.moe_linear(d, x, torch.eye(n, dtype=dt, device="cuda"), None, None, y, None,
                 workspace(M.moe_linear_workspace_size(d)))
    v = z.double()
    f = R.value(fn, v)
    if fn == "silu":
        e = f.abs() * (exp_unit(v.clamp(-104, 104)) + 6 * 2.0 ** -24) + 89 * 2.0 ** -126
    elif fn == "gelu":
        rel = exp_unit(v.clamp(-14, 14) ** 2 / 2) + 5.5e-7 + 8 * 2.0 ** -24
        tail = v.abs() * 0.5 * torch.special.erfc(v.abs() / 2 ** 0.5)
        e = tail * rel + torch.where(v > 0, f * 2.0 ** -23, 0) + 2.0 ** -126
    else:
        e = torch.zeros_like(f)
    for t in (0, T - 1):
        R.check(y[t], (f, e), fn)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("fn", ["silu", "gelu", "relu"])
def test_activation_slopes_over_their_range(fn, dt):
    """In fp32, as the bias gradient of one token with dy = 1. silu, p (1 + z (1 - p)):
    p is off by its quotient's units, 1 - p by p's error and a rounding of p's
    size, which z magnifies. gelu, Phi + z phi: the errors of both terms."""
    z = arguments(dt)[:512].cuda().reshape(1, -1)
    n = z.numel()
    d = M.MoeLinearDims(T=1, N=n, K=8, fn=R.FN[fn], dtype=code(dt), out_f32=1)
    db = empty((n,), F32)
    M.moe_linear_backward(d, torch.ones_like(z), None, None, z, None, None, db,
                          workspace(M.moe_linear_workspace_size(d)))
    v = z.double().reshape(-1)
    s = R.slope(fn, v)
    if fn == "silu":
        p, q = torch.sigmoid(v), torch.sigmoid(-v)
        ep = p * (q * exp_unit(v.clamp(-104, 104)) + 6 * 2.0 ** -24) + 2.0 ** -126
        one = (1 + v * q).abs()
        # 1 - p is exact once p has rounded to 1: then q itself, below 2^-24, is what is lost
        inner = v.abs() * torch.minimum(ep + 2.0 ** -24, q + 2.0 ** -22) + 3 * 2.0 ** -24 * (1 + v.abs() * q)
        e = ep * (one + inner) + p * inner + 2.0 ** -23 * s.abs()
        e = torch.where(v > 60, torch.full_like(e, 2.0 ** -20), e)      # p is 1, the slope 1
    elif fn == "gelu":
        a = v.clamp(-14, 14) ** 2 / 2
        phi = v.abs() * torch.exp(-v * v / 2) / (2 * torch.pi) ** 0.5
        tail = 0.5 * torch.special.erfc(v.abs() / 2 ** 0.5)
        e = phi * (exp_unit(a) + 3 * 2.0 ** -24) + tail * (exp_unit(a) + 5.5e-7 + 8 * 2.0 ** -24) \
            + torch.where(v > 0, 2.0 ** -23, 0.0) + 2.0 ** -23 * s.abs() + 2.0 ** -126
    else:
        e = torch.zeros_like(s)
    R.check(db, (s, e), fn)


# --- waits that run out ---------------------------------------------------------------------

def test_waits_of_the_dense_kernels_run_out():
    """By the clock, through another role's flag, and all alike: bit 2 of the
    status word, long before the seconds that the follower was given."""
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    src = torch.zeros(512, dtype=torch.uint8, device="cuda")
    M.moe_selftest_bounded_wait(status, src, True, 4096)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    M.moe_selftest_bounded_wait(status, None, False, 100)
    end.record()
    torch.cuda.synchronize()
    assert int(status[0]) == M.STATUS_WAIT_TIMEOUT
    assert start.elapsed_time(end) < 1000      # ms; the follower's own limit is 4 s
    assert int(status[1]) == 0


# --- buffers that lie on or beside one another -----------------------------------------------

@pytest.mark.parametrize("save", [M.SAVE_NONE, M.SAVE_16, M.SAVE_8])
@pytest.mark.parametrize("T", [1, 9, 70, 300])
def test_a_block_into_its_own_input(T, save):
    """x is read before y is written: y may be x, with x as the residual or without one."""
    H, I, dt = 520, 1032, BF
    x, wg, wu, wd = ffn_tensors(T, H, I, dt)
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, save=save)
    ws, y = workspace(M.moe_ffn_workspace_size(d)), empty((T, H), dt)
    for residual in (False, True):
        kept = [M.FfnSaved(d) if save else None for _ in range(2)]
        M.moe_ffn(d, x, wg, wu, wd, x if residual else None, y, kept[0], ws)
        inplace = x.clone()
        M.moe_ffn(d, inplace, wg, wu, wd, inplace if residual else None, inplace, kept[1], ws)
        assert torch.equal(inplace, y)
        for n in ("g", "u", "g_s", "u_s", "x_q", "x_s") if save else ():
            a, b = (getattr(k, n) for k in kept)
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b)), n


@pytest.mark.parametrize("T", [1, 30, 300])
def test_slices_of_one_buffer(T):
    """x, residual and y as neighbouring columns."""
    N, K, dt = 264, 136, BF
    x, w, r = rand((T, K), 1, dt, 1), rand((N, K), 0.05, dt, 2), rand((T, N), 1, dt, 4)
    ref = R.linear(x, w, None, r, "none", dt, dt)[0]
    ld = K + 2 * N + 8
    buf = torch.full((T, ld), 7.0, dtype=dt, device="cuda")
    buf[:, :K], buf[:, K:K + N] = x, r
    d = M.MoeLinearDims(T=T, N=N, K=K, ldx=ld, ldr=ld, ldy=ld)
    M.moe_linear(d, buf[:, :K], w, None, buf[:, K:K + N], buf[:, K + N:K + 2 * N], None,
                 workspace(M.moe_linear_workspace_size(d)))
    R.check(buf[:, K + N:K + 2 * N], ref, "y", 1, dt)
    assert torch.equal(buf[:, :K], x) and torch.equal(buf[:, K:K + N], r) and (buf[:, K + 2 * N:] == 7.0).all()


def test_an_overlap_is_an_error_of_the_binding():
    T, H, dt = 30, 264, BF
    x, w = rand((T, H), 1, dt, 1), rand((H, H), 0.05, dt, 2)
    d = M.MoeLinearDims(T=T, N=H, K=H)
    kept = x.clone()
    with pytest.raises(M.MoeError, match="y overlaps x"):
        M.moe_linear(d, x, w, None, x, x, None, workspace(M.moe_linear_workspace_size(d)))
    torch.cuda.synchronize()
    assert torch.equal(x, kept)


# --- order of calls ------------------------------------------------------------------------

@pytest.mark.parametrize("save", [M.SAVE_NONE, M.SAVE_8])
@pytest.mark.parametrize("T", [1, 8, 9, 40, 64, 200])
def test_weights_written_by_the_calls_before_a_block(T, save):
    """wg, wu and wd, each a projection's output, wd the last one before the
    block: other weights every time, so that early reads of them show."""
    H, I, K, dt = 1032, 2056, 1000, BF
    x = rand((T, H), 1, dt, 1)
    dims = [M.MoeLinearDims(T=n, N=k, K=K) for n, k in ((I, H), (I, H), (H, I))]
    ws = workspace(max(M.moe_linear_workspace_size(d) for d in dims))
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, save=save)
    wsf = workspace(M.moe_ffn_workspace_size(d))
    w = [empty((e.T, e.N), dt) for e in dims]
    y = empty((T, H), dt)
    saved = M.FfnSaved(d) if save else None
    parts = [[(rand((e.T, K), 0.2, dt, 10 * i + j), rand((e.N, K), 0.2 / K ** 0.5, dt, 100 + 10 * i + j))
              for j, e in enumerate(dims)] for i in range(4)]
    outs = []
    for _ in range(2):
        for p in parts:
            for e, (a, b), out in zip(dims, p, w):
                M.moe_linear(e, a, b, None, None, out, None, ws)
            M.moe_ffn(d, x, *w, None, y, saved, wsf)
            outs.append(y.clone())
    # the same in a graph
    held = [torch.empty_like(y) for _ in parts]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p, h in zip(parts, held):
            for e, (a, b), out in zip(dims, p, w):
                M.moe_linear(e, a, b, None, None, out, None, ws)
            M.moe_ffn(d, x, *w, None, y, saved, wsf)
            h.copy_(y)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(h, o) for h, o in zip(held, outs))
    del graph
    for i, p in enumerate(parts):
        exact = [R.linear(a, b, None, None, "none", dt, dt)[0][0].to(dt) for a, b in p]
        for e, (a, b), out in zip(dims, p, w):
            M.moe_linear(e, a, b, None, None, out, None, ws)
            torch.cuda.synchronize()
        assert all(((o.double() - v.double()).norm() <= 2 * R.unit(dt) * v.double().norm()) for o, v in zip(w, exact))
        ref = R.ffn(x, *w, None, "silu", dt, dt)[0]
        for o in (outs[i], outs[i + len(parts)]):
            R.check(o, ref, "y", 2, dt)


def test_two_streams_give_what_one_gives():
    """Forward and backward on two streams at once: the bits of the same calls made alone."""
    H, I, dt = 520, 1032, BF
    for T in (1, 9, 30, 100, 400):
        x, wg, wu, wd = ffn_tensors(T, H, I, dt)
        dy = rand((T, H), 0.3, dt, 6)
        d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, save=M.SAVE_16)

        def buffers():
            return M.FfnSaved(d), empty((T, H), dt), ffn_buffers(T, H, I, dt), workspace(M.moe_ffn_workspace_size(d))

        def step(saved, y, got, ws, stream=None):
            M.moe_ffn(d, x, wg, wu, wd, None, y, saved, ws, stream=stream)
            M.moe_ffn_backward(d, dy, x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws,
                               stream=stream)

        alone = buffers()
        step(*alone)
        torch.cuda.synchronize()
        runs = [(torch.cuda.Stream(), buffers()) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(4):
            for s, b in runs:
                step(*b, stream=s)
        torch.cuda.synchronize()
        for _, b in runs:
            assert torch.equal(b[1], alone[1])
            for n in alone[2]:
                assert torch.equal(b[2][n], alone[2][n]), n


# --- offsets past 32 bits in the gated block and the backward passes ---------------------------

def test_linear_gradient_offsets_past_32_bits():
    """65536 x 65536 output gradients: dx by rows, dw and db by columns."""
    T = N = 65536
    K, dt = 16, BF
    x, w, dy, pre = rand((T, K), 1, dt, 1), rand((N, K), 0.3, dt, 2), rand((T, N), 0.01, dt, 3), rand((T, N), 1.5, dt, 4)
    d = M.MoeLinearDims(T=T, N=N, K=K, fn=1)
    dx, dw, db = empty((T, K), dt), empty((N, K), dt), empty((N,), dt)
    M.moe_linear_backward(d, dy, x, w, pre, dx, dw, db, workspace(M.moe_linear_workspace_size(d)))
    for r0 in (0, 32760, 65500):
        part = slice(r0, r0 + 36)
        ref = R.linear_grads(dy[part], x[part], w, pre[part], "silu", False, dt, dt)
        R.check(dx[part], ref["dx"], "dx")
        ref = R.linear_grads(dy[:, part], x, w[part], pre[:, part], "silu", True, dt, dt)
        R.check(dw[part], ref["dw"], "dw")
        R.check(db[part], ref["db"], "db")


@pytest.mark.parametrize("save", [M.SAVE_16, M.SAVE_8])
def test_ffn_offsets_past_32_bits(save):
    """65536 tokens of 65536 hidden elements, forward and backward."""
    T = I = 65536
    H, dt = 16, BF
    x, wg, wu, wd = (rand((T, H), 1, dt, 1), rand((I, H), 0.3, dt, 2), rand((I, H), 0.3, dt, 3),
                     rand((H, I), 0.01, dt, 4))
    dy = rand((T, H), 0.3, dt, 6)
    d = M.MoeFfnDims(T=T, H=H, I=I, fn=1, save=save)
    ws, saved = workspace(M.moe_ffn_workspace_size(d)), M.FfnSaved(d)
    y, got = empty((T, H), dt), ffn_buffers(T, H, I, dt)
    M.moe_ffn(d, x, wg, wu, wd, None, y, saved, ws)
    M.moe_ffn_backward(d, dy, x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], ws)
    for r0 in (0, 32768, 65504):
        part = slice(r0, r0 + 32)
        R.check(y[part], R.ffn(x[part], wg, wu, wd, None, "silu", dt, dt)[0], "y")
        g, u = saved.g[part], saved.u[part]
        gc, uc = saved.g[:, part], saved.u[:, part]
        if save == M.SAVE_8:
            block = slice(r0 // 32, r0 // 32 + 1)
            g, u = R.unpack8(g, saved.g_s[part]), R.unpack8(u, saved.u_s[part])
            gc, uc = R.unpack8(gc, saved.g_s[:, block]), R.unpack8(uc, saved.u_s[:, block])
        ref = R.ffn_grads(dy[part], x[part], wg, wu, wd, g, u, "silu", dt, dt)
        R.check(got["dx"][part], ref["dx"], "dx")
        ref = R.ffn_grads(dy, x, wg[part], wu[part], wd[:, part], gc, uc, "silu", dt, dt)
        R.check(got["dwg"][part], ref["dwg"], "dwg")
        R.check(got["dwu"][part], ref["dwu"], "dwu")
        R.check(got["dwd"][:, part], ref["dwd"], "dwd")
