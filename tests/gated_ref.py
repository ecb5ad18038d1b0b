"""Plain 64-bit forms of a gated recurrent block's operators (gated linear recurrence, gated
feed-forward half, projection in 8-bit integers), in torch on the CPU or the GPU, and the rounding bounds their tests use."""
import math

import torch

from block_ref import U, HALF, act, act_grad, check, sum_depth      # noqa: F401
# check: |got - ref| <= tol + half a step of got's type

CHUNK = 64


# ------------------------------------------------------- gated linear recurrence
def walk(a, b, h0):
    """h_t = a_t h_(t-1) + b_t along dim 1 (B, L, D), step by step within runs of about
    sqrt(L) steps, then over the runs.  A decay of 0 drops what is not finite."""
    bt, l, d = a.shape
    n = max(1, math.isqrt(l))
    runs = -(-l // n)
    pad = runs * n - l
    if pad:
        a = torch.cat([a, torch.ones(bt, pad, d, dtype=a.dtype, device=a.device)], 1)
        b = torch.cat([b, torch.zeros(bt, pad, d, dtype=a.dtype, device=a.device)], 1)
    a, b = a.reshape(bt, runs, n, d), b.reshape(bt, runs, n, d)

    def step(a, h, b):
        return torch.where(a == 0, b, a * h + b)
    h, p = [b[:, :, 0]], [a[:, :, 0]]
    for t in range(1, n):
        h.append(step(a[:, :, t], h[-1], b[:, :, t]))
        p.append(a[:, :, t] * p[-1])
    h, p = torch.stack(h, 2), torch.stack(p, 2)
    first = [h0]
    for k in range(runs - 1):
        first.append(step(p[:, k, -1], first[-1], h[:, k, -1]))
    h = step(p, torch.stack(first, 1)[:, :, None].expand_as(p), h)
    return h.reshape(bt, runs * n, d)[:, :l]


def softplus(v):
    return torch.logaddexp(v, torch.zeros((), dtype=v.dtype, device=v.device))


class Rec:
    """Forward and backward of the recurrence in 64 bits, with bounds of fp32 rounding.

    Relative errors of the parts: sigmoid(v) 6 U + 2 |v| U (exp2 of a rounded product,
    reciprocal), log a 10 U more (softplus, decay, product), a - 1 another 24 U (a - 1 from
    a rounded to 2^-24 where 1 - a >= 0.049), sqrt(1 - a^2) 4 U more.  A step of the state
    and the joins of stretches round by 8 U of the states at either end.
    Underflow: sigmoid(r) and log a below 2^-126 become 0, which moves y = -log a by at most
    t = (c softplus(lam) + 1) 2^-126, and sqrt(1 - a^2) <= sqrt(2 y) by at most sqrt(2 t)
    (sqrt(y + t) - sqrt(y) <= sqrt(t)); y / sqrt(1 - a^2), about sqrt(y / 2), by less."""

    def __init__(self, x, r, i, lam, z=None, h0=None, starts=None, lengths=None, decay=8.0):
        f = torch.float64
        dev = x.device
        bt, l, d = x.shape
        self.x, self.r, self.i = x.to(f), r.to(f), i.to(f)
        self.z = None if z is None else z.to(f)
        self.lam, self.decay = lam.to(f), decay
        self.live = torch.ones(bt, l, 1, dtype=torch.bool, device=dev)
        if lengths is not None:
            self.live = torch.arange(l, device=dev).view(1, l, 1) < lengths.view(bt, 1, 1)
        keep = torch.ones(bt, l, 1, dtype=torch.bool, device=dev)
        if starts is not None:
            keep = (starts == 0).unsqueeze(2)
        zero = torch.zeros((), dtype=f, device=dev)
        one = torch.ones((), dtype=f, device=dev)

        def inside(v):
            return torch.where(self.live, v, zero)
        self.inside = inside
        self.x, self.r, self.i = inside(self.x), inside(self.r), inside(self.i)
        if self.z is not None:
            self.z = inside(self.z)
        self.sr, self.si = torch.sigmoid(self.r), torch.sigmoid(self.i)
        self.la = -decay * softplus(self.lam) * self.sr
        self.a = self.la.exp()
        self.beta = (-torch.expm1(2 * self.la)).sqrt()
        self.g = self.beta * self.si * self.x
        self.h0 = torch.zeros(bt, d, dtype=f, device=dev) if h0 is None else h0.to(f)
        self.carry = torch.where(self.live, torch.where(keep, self.a, zero), one)
        self.h = walk(self.carry, inside(self.g), self.h0)
        self.before = torch.cat([self.h0[:, None], self.h[:, :-1]], 1)
        self.hk = torch.where(keep, self.before, zero)         # 0 at a start
        # bounds
        self.e_sr, self.e_si = U * (6 + 2 * self.r.abs()), U * (6 + 2 * self.i.abs())
        self.e_la = self.e_sr + 10 * U
        self.e_E = self.e_la + 24 * U
        self.e_b = self.e_E + 4 * U
        self.under = (2 * (decay * softplus(self.lam) + 1) * 2.0 ** -126).sqrt()
        self.da = -torch.expm1(self.la) * self.e_E + 2 * U * self.a
        err = (self.hk.abs() * self.da + self.g.abs() * (self.e_b + self.e_si + 3 * U)
               + (self.si * self.x).abs() * self.under
               + 8 * U * (self.h.abs() + self.hk.abs()))
        self.tol_h = walk(self.carry, inside(err), torch.zeros_like(self.h0))
        self.tol_before = torch.cat([torch.zeros_like(self.h0)[:, None], self.tol_h[:, :-1]], 1)

    def fwd(self):
        """(y, h_last, states, and their bounds)."""
        y, tol = self.h, self.tol_h
        if self.z is not None:
            s = self.z * torch.sigmoid(self.z)
            y = self.h * s
            tol = tol * s.abs() + y.abs() * U * (10 + 2 * self.z.abs())
        at = [t - 1 for t in range(0, self.h.shape[1], CHUNK)]
        st = torch.stack([self.h0 if t < 0 else self.h[:, t] for t in at], 1)
        ts = torch.stack([0 * self.h0 if t < 0 else self.tol_h[:, t] for t in at], 1)
        return (self.inside(y), self.h[:, -1], st, self.inside(tol) + 1e-30, self.tol_h[:, -1] + 1e-30,
                ts + 1e-30)

    def bwd(self, dy, dh_last=None):
        """Two dicts: dx, dr, di, dz, dlam, dh0, and their bounds."""
        dy = self.inside(dy.to(torch.float64))
        v, dv = dy, torch.zeros_like(dy)
        if self.z is not None:
            sz = torch.sigmoid(self.z)
            v = dy * self.z * sz
            dv = v.abs() * U * (10 + 2 * self.z.abs())
        last = torch.zeros_like(self.h0) if dh_last is None else dh_last.to(torch.float64)
        back = torch.cat([torch.ones_like(self.h0)[:, None], self.carry[:, 1:].flip(1)], 1)
        u = walk(back, v.flip(1), last).flip(1)
        after = torch.cat([u[:, 1:], last[:, None]], 1)
        da1 = torch.cat([self.inside(self.da)[:, 1:], torch.zeros_like(last)[:, None]], 1)
        tol_u = walk(back, (dv + after.abs() * da1 + 8 * U * (u.abs() + after.abs())).flip(1),
                     torch.zeros_like(last)).flip(1)
        dh0 = self.carry[:, 0] * u[:, 0]
        t_dh0 = (self.carry[:, 0] * tol_u[:, 0] + u[:, 0].abs() * (self.da[:, 0] + 8 * U))
        u, tol_u = self.inside(u), self.inside(tol_u)
        b, si, sr, x, la, a = self.beta, self.si, self.sr, self.x, self.la, self.a
        zero = torch.zeros((), dtype=torch.float64, device=x.device)
        out, tol = {"dh0": dh0}, {"dh0": t_dh0}
        out["dx"] = u * b * si
        tol["dx"] = (tol_u * b * si + out["dx"].abs() * (self.e_b + self.e_si + 4 * U)
                     + (u * si).abs() * self.under)
        ci = torch.sigmoid(-self.i)
        out["di"] = out["dx"] * x * ci
        tol["di"] = (tol["dx"] * (x * ci).abs() + (out["dx"] * x).abs() * (si * self.e_si + U)
                     + 4 * U * out["di"].abs())
        lb = torch.where(b > 0, la / b, zero)
        gx = si * x
        t1, t2 = a * self.hk * la, a * a * lb * gx
        dl = u * (t1 - t2)
        e = (t1.abs() * (self.e_la + 4 * U) + (self.hk * la).abs() * self.da
             + (a * la).abs() * torch.where(self.hk == 0, zero, self.tol_before)
             + t2.abs() * (self.e_la + self.e_b + self.e_si + 8 * U)
             + (lb * gx).abs() * (2 * b * b * self.e_b + 2 * U) + gx.abs() * self.under)
        t_dl = tol_u * (t1.abs() + t2.abs()) + u.abs() * e + 4 * U * dl.abs()
        cr = torch.sigmoid(-self.r)
        out["dr"] = dl * cr
        tol["dr"] = t_dl * cr + dl.abs() * (sr * self.e_sr + U) + 4 * U * out["dr"].abs()
        # d la / d lam = la sigmoid(lam) / softplus(lam)
        k = torch.where(softplus(self.lam) > 0, torch.sigmoid(self.lam) / softplus(self.lam), 1 + zero)
        out["dlam"] = dl.sum((0, 1)) * k
        # a lane adds runs of 64 terms, the runs, 16 stretches, then the workgroups' sums
        bt, l, _ = x.shape
        depth = 64 + l / 1024 + 40 + bt * l / 512 / 4
        tol["dlam"] = (t_dl.sum((0, 1)) + U * depth * dl.abs().sum((0, 1))) * k + 20 * U * out["dlam"].abs()
        if self.z is not None:
            zz, sz = self.z, torch.sigmoid(self.z)
            slope = sz * (1 + zz * torch.sigmoid(-zz))
            out["dz"] = dy * self.h * slope
            tol["dz"] = (dy * slope).abs() * self.tol_h + (dy * self.h).abs() * U * (
                8 + 4 * zz.abs() + 2 * zz * zz)
        return out, {n: t + 1e-30 for n, t in tol.items()}


# ------------------------------------------------- gated feed-forward half
def _act_err(v):
    """Rounding of act(v) and act'(v) at a given v (the functions: a few roundings of v and
    of the result)."""
    return U * (8 + 4 * v.abs() + 2 * v * v)


def glu_fwd(x, w, bias, name):
    """(y, pre, tol_y, tol_pre), float64, of x (M, K) and w (2 F, K)."""
    xd, wd = x.double(), w.double()
    pre = xd @ wd.t()
    tol = U * sum_depth(x.shape[1], x.dtype) * (xd.abs() @ wd.abs().t())
    if bias is not None:
        pre = pre + bias.double()
    tol = tol + U * pre.abs()
    (gate, up), (tg, tu) = pre.chunk(2, 1), tol.chunk(2, 1)
    a = act(name, gate)
    ta = tg if name == "none" else 1.13 * tg + _act_err(gate)      # |act'| < 1.13
    y = a * up
    return y, pre, ta * (up.abs() + tu) + a.abs() * tu + 2 * U * y.abs(), tol


def glu_bwd(x, w, dy, pre, name, grad_dtype):
    """(dx, dw, dbias, tol_dx, tol_dw, tol_db), float64.  Bounds: d's own rounding, what the
    products see of it (2^-8 of it with bf16 gradients of bf16 operands, 2^-16 with fp32
    ones), and the contractions'."""
    dt = w.dtype
    xd, wd, d0 = x.double(), w.double(), dy.double()
    gate, up = pre.double().chunk(2, 1)
    d = torch.cat([d0 * up * act_grad(name, gate), d0 * act(name, gate)], 1)
    fn = torch.cat([(d0 * up).abs() * _act_err(gate), d0.abs() * _act_err(gate)], 1) + 3 * U * d.abs()
    seen = 0.0
    if dt == torch.bfloat16:
        seen = 2.0 ** -16 if grad_dtype == torch.float32 else HALF[dt]
    err = fn + seen * d.abs()
    a = d.abs() + err
    dx, dw, db = d @ wd, d.t() @ xd, d.sum(0)
    tol_dx = err @ wd.abs() + U * sum_depth(w.shape[0], dt) * (a @ wd.abs())
    tol_dw = err.t() @ xd.abs() + U * sum_depth(x.shape[0], dt) * (a.t() @ xd.abs())
    # a column sum: runs of 64 rows, the runs of a chunk, at most a quarter of 2048 chunks
    rows = x.shape[0]
    depth = min(rows, 64) + rows / 256 + 520
    return dx, dw, db, tol_dx, tol_dw, fn.sum(0) + depth * U * a.sum(0)


# ------------------------------------------------- 8-bit integers
def q8_pack(x):
    """(q, s) by exact integer arithmetic in 64 bits: q = round(127 x / max), ties to even, by
    comparing 2 * 127 |x| with odd multiples of max."""
    d = x.double()
    top = d.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    m = torch.where(fine & (top > 0), top, torch.ones_like(top))
    v = torch.where(fine, d.abs(), torch.zeros_like(d))
    f = torch.floor(127.0 * v / m)
    f = torch.where(127.0 * v < f * m, f - 1, f)
    f = torch.where(127.0 * v >= (f + 1) * m, f + 1, f)
    a, b = 254.0 * v, (2 * f + 1) * m
    f = f + ((a > b) | ((a == b) & (f % 2 == 1)))
    q = torch.where(d < 0, -f, f).to(torch.int8)
    # (by a tensor: torch multiplies by the rounded reciprocal of a plain number)
    s = (torch.where(fine, top, torch.full_like(top, math.nan)) / torch.full_like(top, 127.0))[..., 0].float()
    return q, s


def q8_linear(x, w, bias, residual, name):
    """(y, tol) of packed x and w, float64: the sums are exact, the epilogue rounds."""
    (xq, xs), (wq, ws) = x, w
    v = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    tol = 3 * U * v.abs()                    # the sum to fp32, both scales
    if bias is not None:
        v = v + bias.double()
        tol = tol + U * v.abs()
    y = act(name, v)
    if name != "none":
        tol = 1.13 * tol + _act_err(v)
    if residual is not None:
        y = y + residual.double()
        tol = tol + U * y.abs()
    return y, tol
