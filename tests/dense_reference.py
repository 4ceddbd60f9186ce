"""Plain fp64 forms of the dense operators, with error bounds for kernels that
round as the library says it does.

Bounds. u = half a unit of the 16-bit type relative to the value (bf16 2^-8,
f16 2^-11). A product of 16-bit values is exact in fp32; a tensor-core sum
over K adds 16 products at a time to an fp32 accumulator, each addition off by
at most 2^-23 of the running magnitude, which never exceeds S = sum |a||b|: a
sum is within (K/16 + 8) 2^-23 S of the exact one (the 8 covers the epilogue's
few fp32 operations and the partial sums of a split). fp32 activations are
within 2^-20 relative, slopes of f at most 1.2, |f(z)| <= |z|.
Rounded intermediates (h, dz, dg, du) add u |value|, carried through the next
product by sum |error| |weight|.
"""
import math

import torch

FN = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
F16_TINY = 2.0 ** -24       # f16's smallest subnormal; half of it bounds its rounding below 2^-14


def unit(dt):
    return torch.finfo(dt).eps / 2


def value(fn, z):
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if fn == "relu":
        return z.clamp(min=0)
    return z.clone()


def slope(fn, z):
    if fn == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if fn == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if fn == "relu":
        return (z > 0).double()
    return torch.ones_like(z)


def product(a, ea, b, K=None):
    """a [M, K] (off by at most ea) times b [N, K]^T: the product and its bound."""
    K = a.shape[1] if K is None else K
    p = a @ b.t()
    S = a.abs() @ b.abs().t()
    e = (K / 16 + 8) * 2.0 ** -23 * S
    if ea is not None:
        e = e + ea @ b.abs().t()
    return p, e


def stored(v, e, dt):
    """Bound of v (off by e) once it is rounded to dt."""
    if dt is torch.float32:
        return e + 2.0 ** -23 * v.abs()
    tiny = F16_TINY / 2 if dt is torch.float16 else 0.0
    return e + unit(dt) * (v.abs() + e) + tiny


def activated(fn, z, e):
    f = value(fn, z)
    return f, 1.2 * e + 2.0 ** -20 * (z.abs() + f.abs())


def linear(x, w, bias, residual, fn, dt, out):
    z, e = product(x.double(), None, w.double())
    if bias is not None:
        z = z + bias.double()
    pre = (z, stored(z, e, dt))
    y, e = activated(fn, z, e)
    if residual is not None:
        y = y + residual.double()
    return (y, stored(y, e, out)), pre


def gated_hidden(x, wg, wu, fn):
    g, eg = product(x.double(), None, wg.double())
    u, eu = product(x.double(), None, wu.double())
    f, ef = activated(fn, g, eg)
    return g, eg, u, eu, f * u, ef * u.abs() + f.abs() * eu + ef * eu


def ffn(x, wg, wu, wd, residual, fn, dt, out):
    g, eg, u, eu, h, eh = gated_hidden(x, wg, wu, fn)
    y, e = product(h, stored(h, eh, dt), wd.double())
    if residual is not None:
        y = y + residual.double()
    return (y, stored(y, e, out)), (g, eg), (u, eu)


def linear_grads(dy, x, w, pre, fn, bias, dt, out):
    dz, e = dy.double(), None
    if fn != "none":
        d = slope(fn, pre.double())
        ed = 2.0 ** -20 * dz.abs() * (d.abs() + pre.double().abs())
        dz = dz * d
        e = stored(dz, ed, dt)
    else:
        ed = torch.zeros_like(dz)
    T = dy.shape[0]
    dx, ex = product(dz, e, w.double().t())
    dw, ew = product(dz.t(), None if e is None else e.t(), x.double().t(), T)
    r = {"dx": (dx, stored(dx, ex, out)), "dw": (dw, stored(dw, ew, out))}
    if bias:
        db = dz.sum(0)
        eb = ed.sum(0) + (T + 8) * 2.0 ** -23 * dz.abs().sum(0)
        r["db"] = (db, stored(db, eb, out))
    return r


def ffn_grads(dy, x, wg, wu, wd, g, u, fn, dt, out):
    """From the values g, u (exact inputs here) of the saved activations."""
    T = dy.shape[0]
    g, u, dy, x = g.double(), u.double(), dy.double(), x.double()
    dh, e = product(dy, None, wd.double().t())
    f, s = value(fn, g), slope(fn, g)
    small = 2.0 ** -20
    dg, du, h = dh * u * s, dh * f, f * u
    edg = stored(dg, (e * s.abs() + small * dh.abs() * (s.abs() + g.abs())) * u.abs(), dt)
    edu = stored(du, e * f.abs() + small * dh.abs() * (f.abs() + g.abs()), dt)
    eh = stored(h, small * (f.abs() + g.abs()) * u.abs(), dt)
    a, ea = product(dg, edg, wg.double().t())
    b, eb = product(du, edu, wu.double().t())
    dx = a + b
    r = {"dx": (dx, stored(dx, ea + eb + 2.0 ** -20 * (a.abs() + b.abs()), out))}
    for n, v, ev, o in (("dwg", dg, edg, x), ("dwu", du, edu, x)):
        p, ep = product(v.t(), ev.t(), o.t(), T)
        r[n] = (p, stored(p, ep, out))
    p, ep = product(h.t(), eh.t(), dy.t(), T)
    r["dwd"] = (p.t(), stored(p, ep, out).t())
    return r


def check(got, ref, name, roundings=None, dt=None):
    """Every element within its bound and, for `roundings` 16-bit roundings on
    the way (each off by at most u/sqrt(3) in the root mean square, independent
    of one another), the whole within their root sum of squares."""
    v, e = ref
    got = got.double()
    assert got.shape == v.shape, f"{name}: shape"
    err = (got - v).abs()
    bad = ~(err <= e)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements off, first {i}: "
                             f"got {got[i].item()}, want {v[i].item()} +- {e[i].item():.3e}")
    if roundings and v.numel() >= 4096 and v.norm() > 0:
        rel = ((got - v).norm() / v.norm()).item()
        bound = unit(dt) * math.sqrt(roundings / 3) + 2.0 ** -16
        assert rel <= bound, f"{name}: root mean square error {rel:.3e} above {bound:.3e}"


# --- 8-bit checkpoints ------------------------------------------------------------

def e4m3_table():
    """The value of every E4M3 code, by its fields (0x7F and 0xFF are NaN)."""
    t = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = math.nan
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (1 + m / 8) * 2.0 ** (e - 7)
        t.append(-v if s else v)
    return t


def pack8(x):
    """Codes and scales of x [rows, cols] (fp64 on the CPU), element by element of the definition."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    mags = torch.tensor(e4m3_table()[:127], dtype=torch.float64)
    q = torch.zeros(rows, cols, dtype=torch.uint8)
    s = torch.zeros(rows, nb, dtype=torch.uint8)
    for b in range(nb):
        v = x[:, 32 * b:32 * b + 32]
        for r in range(rows):
            a = v[r].abs().max().item() if not torch.isnan(v[r]).any() else math.nan
            if not math.isfinite(a):
                s[r, b] = 255
                continue
            X = -127
            while a > 448 * 2.0 ** X:
                X += 1
            s[r, b] = X + 127
            y = v[r] * 2.0 ** -X
            d = (y.abs().unsqueeze(1) - mags).abs()
            best = d.min(dim=1, keepdim=True).values
            near = d == best                                 # one code, or two at a tie
            idx = torch.arange(127)
            pick = torch.where(near & (idx % 2 == 0), idx, torch.where(near & (near.sum(1, keepdim=True) == 1), idx, -1))
            code = pick.max(dim=1).values
            q[r, 32 * b:32 * b + v.shape[1]] = (code + 128 * torch.signbit(v[r]).long()).to(torch.uint8)
    return q, s


def unpack8(q, s):
    """fp64 values of codes and scales (any device)."""
    t = torch.tensor(e4m3_table(), dtype=torch.float64, device=q.device)
    sc = torch.exp2(s.double() - 127)
    sc = torch.where(s == 255, torch.full_like(sc, math.nan), sc)
    return t[q.long()] * sc.repeat_interleave(32, dim=1)[:, :q.shape[1]]


def scale8(a):
    """Scale codes of blocks whose largest magnitudes are a (fp64)."""
    m, e = torch.frexp(a / 448)
    return (torch.where(m == 0.5, e - 1, e) + 127).clamp(0, 254)


def codes8(v, s):
    """Magnitude codes of v [rows, cols] under the scale codes s, nearest (ties are not looked after)."""
    mags = torch.tensor(e4m3_table()[:127], dtype=torch.float64, device=v.device)
    sc = torch.exp2(127 - s.double()).repeat_interleave(32, dim=1)[:, :v.shape[1]]
    return torch.bucketize(v * sc, (mags[1:] + mags[:-1]) / 2)


def check_codes(v, rel, q, s, name):
    """Codes q and scales s of values known to be within rel of v (fp64, all
    positive): wherever no border of the grid lies that close, the code is v's.
    Returns how many elements that holds for."""
    top = torch.nn.functional.pad(v, (0, -v.shape[1] % 32)).reshape(v.shape[0], -1, 32).amax(-1)
    lo, hi = scale8(top * (1 - rel)), scale8(top * (1 + rel))
    sure = lo == hi
    assert torch.equal(s[sure].long(), lo[sure]), f"{name}: scales"
    lo, hi = codes8(v * (1 - rel), s), codes8(v * (1 + rel), s)
    sure = (lo == hi) & sure.repeat_interleave(32, dim=1)[:, :v.shape[1]]
    off = int((q.long() != lo)[sure].sum())
    assert off == 0, f"{name}: {off} of {int(sure.sum())} codes are off"
    return int(sure.sum())
