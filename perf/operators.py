"""Cases that time the dense operators of the library: the projection with a
fused epilogue (moe_linear), the gated feed-forward block (moe_ffn), both with
their backward passes, and the 8-bit activation checkpoints.

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end) or, with ``own`` set, through the library's
entry points. ``exact`` computes the same outputs in fp64.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_FNS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
_BLOCK = 32          # elements that share one scale of an 8-bit checkpoint
_TOP = 448.0         # largest E4M3 magnitude


def listed():
    return [
        # one token through a narrow projection (a latent layer's down-projection): latency and weight streaming
        dict(name="linear_token", op="linear", T=1, K=7168, N=2048, fn="none", bias=False, residual=False,
             dtype="bf16"),
        # a small decode batch back to the hidden width, added to the residual stream
        dict(name="linear_batch", op="linear", T=16, K=2048, N=7168, fn="none", bias=False, residual=True,
             dtype="bf16"),
        # a prompt through a biased projection to the hidden width, added to the residual stream
        dict(name="linear_prompt", op="linear", T=4096, K=2048, N=8192, fn="none", bias=True, residual=True,
             dtype="bf16"),
        # ragged sizes that no tile divides, in f16, with an activation
        dict(name="linear_ragged", op="linear", T=333, K=1000, N=2056, fn="gelu", bias=True, residual=False,
             dtype="f16"),
        # training step of an activated, biased projection: input, weight and bias gradients
        dict(name="linear_grad", op="linear_grad", T=4096, K=8192, N=2048, fn="silu", bias=True, dtype="bf16"),
        # one token through a gated block of the shared expert's size
        dict(name="ffn_token", op="ffn", T=1, H=8192, I=2048, fn="silu", residual=True, dtype="bf16"),
        # a decode batch through the same block
        dict(name="ffn_batch", op="ffn", T=32, H=8192, I=2048, fn="silu", residual=True, dtype="bf16"),
        # a prompt through the same block
        dict(name="ffn_prompt", op="ffn", T=4096, H=8192, I=2048, fn="silu", residual=True, dtype="bf16"),
        # backward pass of the block from saved 16-bit gate and up projections
        dict(name="ffn_grad", op="ffn_grad", T=4096, H=8192, I=2048, fn="silu", dtype="bf16"),
        # the same in f16 at sizes that no tile divides
        dict(name="ffn_grad_ragged", op="ffn_grad", T=777, H=1000, I=1352, fn="gelu", dtype="f16"),
        # writing a prompt's activations as an 8-bit checkpoint and reading them back
        dict(name="ckpt8_pass", op="ckpt8", T=4096, W=8192, dtype="bf16"),
        # a training step of the block whose saved activations are all held in 8 bits
        dict(name="ffn_step8", op="ffn_step8", T=4096, H=8192, I=2048, fn="silu", dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "ffn", "ffn", "ffn_grad", "ckpt8", "ffn_step8"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    T = _log_int(rng, 1, 4096)
    wide = 8 * _log_int(rng, 16, 1024)
    narrow = 8 * _log_int(rng, 16, 256)
    if op == "linear" or op == "linear_grad":
        if rng.random() < 0.5:
            wide, narrow = narrow, wide
        case = dict(op=op, T=T, K=wide, N=narrow, fn=rng.choice(["none", "none", "silu", "gelu", "relu"]),
                    bias=rng.random() < 0.5, dtype=dtype)
        if op == "linear":
            case["residual"] = rng.random() < 0.5
        return case
    if op == "ckpt8":
        return dict(op=op, T=T, W=wide, dtype=dtype)
    case = dict(op=op, T=T, H=wide, I=narrow, fn=rng.choice(["silu", "silu", "gelu", "relu"]), dtype=dtype)
    if op == "ffn":
        case["residual"] = rng.random() < 0.7
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _inputs(case, seed):
    """The tensors a user has in hand: N(0, 1) activations, N(0, 0.02)
    weights, N(0, 0.05) output gradients, rounded to the case's type."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    s = {}
    op = case["op"]
    if op in ("linear", "linear_grad"):
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = normal((T, K), 1.0)
        s["w"] = normal((N, K), 0.02)
        s["bias"] = normal((N,), 0.5) if case["bias"] else None
        if op == "linear":
            s["residual"] = normal((T, N), 1.0) if case["residual"] else None
        else:
            s["dy"] = normal((T, N), 0.05)
            s["pre"] = None
            if case["fn"] != "none":     # what the forward pass saved
                z = s["x"].float() @ s["w"].float().t()
                s["pre"] = (z + s["bias"].float() if case["bias"] else z).to(dt)
    elif op == "ckpt8":
        # activations whose rows differ in size, as a residual stream's do
        x = torch.randn((case["T"], case["W"]), generator=g, device="cuda")
        x *= torch.exp(torch.randn((case["T"], 1), generator=g, device="cuda"))
        s["x"] = x.to(dt)
    else:
        T, H, I = case["T"], case["H"], case["I"]
        s["x"] = normal((T, H), 1.0)
        s["wg"] = normal((I, H), 0.02)
        s["wu"] = normal((I, H), 0.02)
        s["wd"] = normal((H, I), 0.02)
        if op == "ffn":
            s["residual"] = normal((T, H), 1.0) if case["residual"] else None
        else:
            s["dy"] = normal((T, H), 0.05)
        if op == "ffn_grad":
            s["g"] = (s["x"].float() @ s["wg"].float().t()).to(dt)
            s["u"] = (s["x"].float() @ s["wu"].float().t()).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """Dims, workspace and output buffers that a program keeps between calls."""
    import mxfp4_routed_expert_04_b200 as M

    case = s["case"]
    op = case["op"]
    dt = M.DTYPE_BF16 if case["dtype"] == "bf16" else M.DTYPE_F16
    like = torch.empty_like
    if op in ("linear", "linear_grad"):
        d = M.MoeLinearDims(T=case["T"], N=case["N"], K=case["K"], fn=_FNS[case["fn"]], dtype=dt)
        s["ws"] = torch.empty(M.moe_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
        if op == "linear":
            s["y"] = torch.empty((case["T"], case["N"]), dtype=s["x"].dtype, device="cuda")
        else:
            s["dx"], s["dw"] = like(s["x"]), like(s["w"])
            s["db"] = like(s["bias"]) if case["bias"] else None
    elif op == "ckpt8":
        T, W = case["T"], case["W"]
        s["dt"] = dt
        s["q"] = torch.empty((T, W), dtype=torch.uint8, device="cuda")
        s["s"] = torch.empty((T, (W + _BLOCK - 1) // _BLOCK), dtype=torch.uint8, device="cuda")
        s["y"] = like(s["x"])
        s["M"] = M
        return
    else:
        save = {"ffn": M.SAVE_NONE, "ffn_grad": M.SAVE_16, "ffn_step8": M.SAVE_8}[op]
        d = M.MoeFfnDims(T=case["T"], H=case["H"], I=case["I"], fn=_FNS[case["fn"]], dtype=dt, save=save)
        s["ws"] = torch.empty(M.moe_ffn_workspace_size(d), dtype=torch.uint8, device="cuda")
        if op != "ffn_grad":
            s["y"] = like(s["x"])
        if op == "ffn_grad":
            s["saved"] = M.FfnSaved(d, g=s["g"], u=s["u"])
        elif op == "ffn_step8":
            s["saved"] = M.FfnSaved(d)
        if op != "ffn":
            s["dx"], s["dwg"], s["dwu"], s["dwd"] = like(s["x"]), like(s["wg"]), like(s["wu"]), like(s["wd"])
    s["d"], s["M"] = d, M
    M.moe_dense_workspace_init(s["ws"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    M, op = s["M"], s["case"]["op"]
    if op == "linear":
        M.moe_linear(s["d"], s["x"], s["w"], s["bias"], s["residual"], s["y"], None, s["ws"])
        return s["y"]
    if op == "linear_grad":
        M.moe_linear_backward(s["d"], s["dy"], s["x"], s["w"], s["pre"], s["dx"], s["dw"], s["db"], s["ws"])
        return (s["dx"], s["dw"]) if s["db"] is None else (s["dx"], s["dw"], s["db"])
    if op == "ffn":
        M.moe_ffn(s["d"], s["x"], s["wg"], s["wu"], s["wd"], s["residual"], s["y"], None, s["ws"])
        return s["y"]
    if op == "ffn_grad":
        M.moe_ffn_backward(s["d"], s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["saved"], s["dx"], s["dwg"],
                           s["dwu"], s["dwd"], s["ws"])
        return s["dx"], s["dwg"], s["dwu"], s["dwd"]
    if op == "ckpt8":
        M.moe_ckpt8_pack(s["x"], s["q"], s["s"])
        M.moe_ckpt8_unpack(s["q"], s["s"], s["y"])
        return s["y"]
    # a step: the forward pass keeps x, g and u in 8 bits, the backward pass reads nothing else of them
    M.moe_ffn(s["d"], s["x"], s["wg"], s["wu"], s["wd"], None, s["y"], s["saved"], s["ws"])
    M.moe_ffn_backward(s["d"], s["dy"], None, s["wg"], s["wu"], s["wd"], s["saved"], s["dx"], s["dwg"],
                       s["dwu"], s["dwd"], s["ws"])
    return s["y"], s["dx"], s["dwg"], s["dwu"], s["dwd"]


def _fn(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "relu":
        return torch.clamp(z, min=0)
    return z


def _dfn(name, z):
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _through_8_bits(x):
    """x (fp32) as an 8-bit checkpoint holds it: per 32 elements of a row the
    smallest power of two that brings the largest magnitude to 448 or below,
    elements rounded to E4M3 (ties to even)."""
    T, W = x.shape
    pad = -W % _BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).reshape(T, -1, _BLOCK)
    amax = b.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(amax)                         # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(b, -e)
    _, ve = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ve - 1).clamp(min=-6) - 3)
    v = torch.ldexp(torch.round(v / step) * step, e)
    return v.reshape(T, W + pad)[:, :W]


def _ffn_grads(name, dy, x, wg, wu, wd, g, u):
    a, da = _fn(name, g), _dfn(name, g)
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, dy.t() @ (a * u)


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], s["x"].dtype
    x = s["x"].float()
    if op == "ckpt8":
        return _through_8_bits(x).to(dt)
    name = case["fn"]
    if op == "linear":
        z = x @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _fn(name, z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    if op == "linear_grad":
        dz = s["dy"].float()
        if s["pre"] is not None:
            dz = dz * _dfn(name, s["pre"].float())
        out = [dz @ s["w"].float(), dz.t() @ x]
        if s["bias"] is not None:
            out.append(dz.sum(dim=0))
        return tuple(o.to(dt) for o in out)
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    if op == "ffn_grad":
        out = _ffn_grads(name, s["dy"].float(), x, wg, wu, wd, s["g"].float(), s["u"].float())
        return tuple(o.to(dt) for o in out)
    g, u = x @ wg.t(), x @ wu.t()
    y = (_fn(name, g) * u) @ wd.t()
    if op == "ffn":
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    out = _ffn_grads(name, s["dy"].float(), _through_8_bits(x), wg, wu, wd, _through_8_bits(g),
                     _through_8_bits(u))
    return (y.to(dt),) + tuple(o.to(dt) for o in out)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op in ("linear", "linear_grad"):
        N, K = case["N"], case["K"]
        if op == "linear":
            n = T * K + N * K + T * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)
            return {"bytes": 2 * n, "flops": 2 * T * N * K}
        n = 2 * T * K + 2 * N * K + T * N * (1 if case["fn"] == "none" else 2) + (N if case["bias"] else 0)
        return {"bytes": 2 * n, "flops": 4 * T * N * K}
    if op == "ckpt8":
        W = case["W"]
        held = T * W + T * ((W + _BLOCK - 1) // _BLOCK)
        return {"bytes": 4 * T * W + 2 * held, "flops": 4 * T * W}
    H, I = case["H"], case["I"]
    mac = T * H * I
    if op == "ffn":
        return {"bytes": 2 * (T * H * (3 if case["residual"] else 2) + 3 * H * I), "flops": 6 * mac}
    if op == "ffn_grad":
        return {"bytes": 2 * (3 * T * H + 2 * T * I + 6 * H * I), "flops": 12 * mac}
    held = sum(T * n + T * ((n + _BLOCK - 1) // _BLOCK) for n in (H, I, I))
    return {"bytes": 2 * (4 * T * H + 6 * H * I) + 2 * held, "flops": 18 * mac}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _value_slope(name, z):
    """f(z) and f'(z) of the activation, fp64."""
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1.0 - p)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z.square() / 2.0) * (0.5 * math.sqrt(2.0 / math.pi))
    if name == "relu":
        on = z > 0
        return torch.where(on, z, 0.0), on.double()
    return z, torch.ones_like(z)


def _held_in_8(x):
    """fp64 values -> the values an 8-bit checkpoint holds, by a search of the
    E4M3 grid: the magnitudes k/8 * 2^j (8 <= k < 16, j >= -6) and k * 2^-9."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    for c in range(0, cols, _BLOCK):
        b = x[:, c:c + _BLOCK]
        top = b.abs().amax(dim=1, keepdim=True)
        ex = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / _TOP))
        ex = torch.where(top > _TOP * torch.exp2(ex), ex + 1, ex)
        ex = torch.where(top <= _TOP * torch.exp2(ex - 1), ex - 1, ex).clamp(-127, 127)
        q = b / torch.exp2(ex)
        low = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
        low = torch.where(torch.exp2(low) > q.abs().clamp(min=2.0 ** -6), low - 1, low)
        low = torch.where(torch.exp2(low + 1) <= q.abs(), low + 1, low)
        unit = torch.exp2(low - 3)
        out[:, c:c + _BLOCK] = torch.round(q / unit) * unit * torch.exp2(ex)
    return out


def exact(case, seed):
    t = _inputs(case, seed)
    op = case["op"]
    t = {k: (v.double() if v is not None else None) for k, v in t.items()}
    if op == "ckpt8":
        return _held_in_8(t["x"])
    name = case["fn"]
    if op == "linear":
        z = torch.einsum("tk,nk->tn", t["x"], t["w"])
        if t["bias"] is not None:
            z += t["bias"]
        y = _value_slope(name, z)[0]
        return y if t["residual"] is None else t["residual"] + y
    if op == "linear_grad":
        dz = t["dy"] if t["pre"] is None else _value_slope(name, t["pre"])[1] * t["dy"]
        out = (torch.einsum("tn,nk->tk", dz, t["w"]), torch.einsum("tn,tk->nk", dz, t["x"]))
        return out if t["bias"] is None else out + (torch.einsum("tn->n", dz),)
    if op == "ffn_grad":
        gate, up, y = t["g"], t["u"], None
        x = t["x"]
    else:
        gate = torch.einsum("th,ih->ti", t["x"], t["wg"])
        up = torch.einsum("th,ih->ti", t["x"], t["wu"])
        y = torch.einsum("ti,hi->th", _value_slope(name, gate)[0] * up, t["wd"])
        if op == "ffn":
            return y if t["residual"] is None else t["residual"] + y
        x, gate, up = _held_in_8(t["x"]), _held_in_8(gate), _held_in_8(up)
    value, slope = _value_slope(name, gate)
    dh = torch.einsum("th,hi->ti", t["dy"], t["wd"])
    dgate, dup = slope * up * dh, value * dh
    grads = (torch.einsum("ti,ih->th", dgate, t["wg"]) + torch.einsum("ti,ih->th", dup, t["wu"]),
             torch.einsum("ti,th->ih", dgate, x), torch.einsum("ti,th->ih", dup, x),
             torch.einsum("th,ti->hi", t["dy"], value * up))
    return grads if y is None else (y,) + grads
