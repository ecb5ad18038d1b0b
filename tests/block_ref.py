"""Plain 64-bit forms of the operators around the scan (layer norm, linear
projections, 8-bit checkpoints), in torch on the CPU or the GPU, and the
rounding bounds their tests use."""
import math

import numpy as np
import torch

U = 2.0 ** -24                                      # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # finfo(t).eps / 2
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def normal_cdf(v):
    """Phi(v); by erfc, since torch.special.ndtr returns 0 in the far negative tail
    on the GPU (Phi(-12) = 1.8e-33)."""
    return 0.5 * torch.special.erfc(-v * math.sqrt(0.5))


def act(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * normal_cdf(v)
    if name == "softplus":
        return torch.logaddexp(v, torch.zeros((), dtype=v.dtype, device=v.device))
    return v


def act_grad(name, v):
    if name == "silu":
        s = torch.sigmoid(v)
        return s + v * s * torch.sigmoid(-v)
    if name == "gelu":
        return normal_cdf(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "softplus":
        return torch.sigmoid(v)
    return torch.ones_like(v)


def sum_depth(k, dtype):
    """Rounding steps (of 2^-24) on the way of one term through a contraction of
    length k: a bf16 MFMA adds 32 products at a time, in steps that may truncate
    (two half-steps); an fp32 one adds them one by one.  Up to 64 splits and a
    64-term tree are added on top."""
    return 2.0 * (k / 32 + 104) if dtype == torch.bfloat16 else k + 72.0


def norm_fwd(x, residual, weight, bias, eps):
    """(y, sum, mean, rstd, tol_y, tol_mean, tol_rstd) of rows x, all float64;
    the tolerances count fp32 rounding, not the outputs' own."""
    s = x.double() if residual is None else x.double() + residual.double()
    mean = s.mean(-1, keepdim=True)
    var = (s - mean).square().mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    xh = (s - mean) * rstd
    w = torch.ones_like(s[..., :1, :]) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    y = xh * w + b
    # a row sum adds at most 32 values per thread, then 6 + 16 partial sums, and
    # the residual add rounds once: the centred value is off by at most d
    d = U * (56 * s.abs().mean(-1, keepdim=True) + 2 * s.abs().amax(-1, keepdim=True))
    rel = 30 * U + d * rstd                       # of rstd (var: 56 U + 2 d / sigma, halved)
    tol_y = w.abs() * (rstd * d + xh.abs() * rel) + 4 * U * ((xh * w).abs() + b.abs() + y.abs())
    return y, s, mean[..., 0], rstd[..., 0], tol_y, d[..., 0], (rel * rstd)[..., 0]


def norm_bwd(s, dy, mean, rstd, weight, dsum):
    """(dx, dweight, dbias, tol_dx, tol_dw, tol_db), float64, rows in dim 0."""
    s, dy, mean, rstd = s.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones_like(s[:1]) if weight is None else weight.double()
    xh = (s - mean) * rstd
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    tol = rstd * U * (4 * g.abs() + 60 * g.abs().mean(1, keepdim=True) + 4 * m1.abs()
                      + xh.abs() * (64 * (g * xh).abs().mean(1, keepdim=True) + 6 * m2.abs()))
    if dsum is not None:
        dx = dx + dsum.double()
        tol = tol + 2 * U * dsum.double().abs()
    tol = tol + 2 * U * dx.abs()
    # a column sum walks at most rows / 1024 + 1 rows, then a quarter of at most
    # 4096 partial sums, then 3 additions; xh carries 3 roundings
    rows = s.shape[0]
    depth = min(rows + 3, 4096) / 4 + rows / 1024 + 20
    return (dx, (dy * xh).sum(0), dy.sum(0), tol, depth * U * (dy * xh).abs().sum(0),
            depth * U * dy.abs().sum(0))


def linear_fwd(x, w, bias, residual, name):
    """(y, pre, tol_y, tol_pre), float64."""
    dt = x.dtype
    xd, wd = x.double(), w.double()
    pre = xd @ wd.t()
    tol_pre = U * sum_depth(x.shape[1], dt) * (xd.abs() @ wd.abs().t())
    if bias is not None:
        pre = pre + bias.double()
    tol_pre = tol_pre + U * pre.abs()
    y = act(name, pre)
    tol = tol_pre
    if name != "none":      # |act'| < 1.13; the functions: a few roundings of v and of y
        tol = 1.13 * tol_pre + U * (8 * (1 + pre.abs()) + 2 * pre * pre)
    if residual is not None:
        y = y + residual.double()
        tol = tol + U * y.abs()
    return y, pre, tol, tol_pre


def linear_bwd(x, w, dy, pre, name):
    """(dx, dw, dbias, tol_dx, tol_dw, tol_db), float64; x, w, pre of one dtype.
    Bounds: the contraction's, and one rounding of dpre to the operands' type
    unless it is dy itself."""
    dt = w.dtype
    xd, wd = x.double(), w.double()
    d = dy.double()
    e = 0.0
    if name != "none":
        p = pre.double()
        d = d * act_grad(name, p)
        fn = U * (8 + 4 * p.abs() + 2 * p * p) * dy.double().abs()   # act' and the product
    else:
        fn = torch.zeros_like(d)
    if name != "none" or dy.dtype != dt:
        e = HALF[dt]
    err = fn + e * d.abs()
    a = d.abs() + err
    dx, dw, db = d @ wd, d.t() @ xd, d.sum(0)
    tol_dx = err @ wd.abs() + U * sum_depth(w.shape[0], dt) * (a @ wd.abs())
    tol_dw = err.t() @ xd.abs() + U * sum_depth(x.shape[0], dt) * (a.t() @ xd.abs())
    # a column sum: at most a quarter of 1024 chunks after a quarter of a chunk's rows
    rows = x.shape[0]
    depth = rows / 4 + 264
    tol_db = fn.sum(0) + depth * U * a.sum(0)
    return dx, dw, db, tol_dx, tol_dw, tol_db


def ckpt_pack(x):
    """(q, e) of a float32 array (rows, D), by integer arithmetic on the bits."""
    rows, dim = x.shape
    nb = -(-dim // 32)
    xb = np.zeros((rows, nb * 32), np.float32)
    xb[:, :dim] = x
    xb = xb.reshape(rows, nb, 32)
    top = (np.abs(xb).view(np.uint32).max(axis=2) >> 23).astype(np.int64)
    e = np.where(top == 255, 255, np.maximum(1, top - 6))
    with np.errstate(all="ignore"):
        q = np.rint(xb.astype(np.float64) * np.exp2(127.0 - e)[..., None])
    q = np.where((e == 255)[..., None], 0, np.clip(np.nan_to_num(q), -127, 127))
    return q.astype(np.int8).reshape(rows, nb * 32)[:, :dim], e.astype(np.uint8)


def ckpt_unpack(q, e):
    unit = np.where(e == 255, np.nan, np.exp2(e.astype(np.float64) - 127.0))
    return q.astype(np.float64) * np.repeat(unit, 32, axis=1)[:, :q.shape[1]]


def check(got, ref, tol, what):
    """|got - ref| <= tol + half a step of got's type, everywhere."""
    g = got.double()
    bound = tol + HALF[got.dtype] * (ref.abs() + tol) + 1e-37
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert bool(torch.isfinite(g).all()), what + ": non-finite output"
    bad = (g - ref).abs() / bound
    worst = float(bad.max())
    assert worst <= 1.0, "%s: worst error %.3g of its bound" % (what, worst)
    return worst
