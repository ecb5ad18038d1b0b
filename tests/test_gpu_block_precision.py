"""Precision of the operators around the scan where sums are long or operands are
narrower than what they are multiplied with, against 64-bit forms of the same
inputs.  The bounds count rounding steps of the order in which the kernels add."""
import pytest
import torch

from selective_state_space_69_amd import binding as B
import block_ref as ref
from block_ref import DT, U, check
from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    B.load_library()
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.float32, scale=1.0, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + offset).to(dtype)


# ---------------------------------------- fp32 gradients of bf16 operands
# hi = bf16(v) is off by at most 2^-8 |v|, what is left of v is exact in fp32, and lo,
# its bf16, is off by at most 2^-8 of that: the products see v to 2^-16 |v|.
SUM2 = 2.0 ** -16


def bwd_fp32(x, w, dy, pre, name):
    """(dx, dw, tol_dx, tol_dw), float64: twice the terms of a plain contraction
    (hi and lo), of sizes that add up to at most (1 + 2^-7) |v|."""
    d = dy.double()
    err = torch.zeros_like(d)
    if name != "none":
        p = pre.double()
        d = d * ref.act_grad(name, p)
        err = U * (8 + 4 * p.abs() + 2 * p * p) * dy.double().abs()    # act' and the product
    err = err + SUM2 * (d.abs() + err)
    a = (1 + 2.0 ** -7) * (d.abs() + err)
    xd, wd = x.double(), w.double()
    n, m = w.shape[0], x.shape[0]
    tol_dx = err @ wd.abs() + U * ref.sum_depth(2 * n, w.dtype) * (a @ wd.abs())
    tol_dw = err.t() @ xd.abs() + U * ref.sum_depth(2 * m, w.dtype) * (a.t() @ xd.abs())
    return d @ wd, d.t() @ xd, tol_dx, tol_dw


FP32_GRADS = [
    # M, K, N, dy, act, extra columns of x, checkpoint
    (1, 1, 1, "f32", "none", 0, False),
    (1, 64, 40, "bf16", "silu", 0, False),
    (3, 33, 5, "f32", "gelu", 0, False),
    (17, 40, 7, "f32", "none", 0, True),
    (31, 72, 31, "bf16", "softplus", 0, False),
    (32, 96, 33, "f32", "none", 32, False),
    (33, 136, 16, "f32", "silu", 3, False),
    (64, 520, 129, "bf16", "gelu", 0, True),
    (100, 773, 251, "f32", "none", 0, False),
    (129, 128, 128, "bf16", "silu", 8, False),
    (300, 1000, 72, "f32", "softplus", 0, True),
    (520, 4072, 4060, "f32", "none", 0, False),
    (1003, 264, 520, "bf16", "gelu", 0, False),
    (1500, 768, 1536, "f32", "none", 0, False),
    (5003, 768, 1536, "bf16", "silu", 0, False),
    (3001, 770, 1537, "f32", "gelu", 0, False),
    # many rows over few columns, and dx over a contraction of few values
    (40000, 24, 48, "f32", "none", 0, False),
    (8190, 2560, 44, "bf16", "softplus", 32, False),
    (8190, 4090, 37, "f32", "silu", 0, False),
    # 256 x 256 tiles: dx alone, dw alone, both in one launch (the last round of dw
    # reaching some and all of the workgroups, partial last stages)
    (4060, 4072, 520, "f32", "none", 0, False),
    (2600, 4090, 4080, "bf16", "silu", 0, False),
    (9003, 2950, 2901, "f32", "none", 0, True),
    (4096, 4096, 4096, "f32", "softplus", 0, False),
]


@pytest.mark.parametrize("case", FP32_GRADS, ids=lambda c: "m%d_k%d_n%d_%s_%s_x%d_q%d" % c)
def test_fp32_gradients_of_bf16_operands(case):
    """dpre past an activation or from an fp32 dy is not cut to bf16 before the
    products of fp32 gradients."""
    log("fp32 gradients", case)
    m, k, n, td, name, extra, packed = case
    sd = 300 + 10 * FP32_GRADS.index(case)
    x = rand(sd, m, k + extra, dtype=torch.bfloat16, offset=0.1)[:, :k]
    w = rand(sd + 1, n, k, dtype=torch.bfloat16, scale=k ** -0.5)
    dy = rand(sd + 2, m, n, dtype=DT[td])
    pre = rand(sd + 3, m, n, dtype=torch.bfloat16, scale=2.0) if name != "none" else None
    xin = x
    if packed:
        xin = B.ckpt_pack(x)
        x = B.ckpt_unpack(*xin)
    got = B.linear_bwd(xin, w, dy, pre=pre, act=name, bias=True, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    dx, dw, tx, tw = bwd_fp32(x, w, dy, pre, name)
    check(got["dx"], dx, tx, "dx")
    check(got["dw"], dw, tw, "dw")
    one = B.linear_bwd(xin, w, dy, pre=pre, act=name, grad_dtype=torch.float32, need_dx=False)
    assert torch.equal(one["dw"], got["dw"])
    one = B.linear_bwd(None, w, dy, pre=pre, act=name, grad_dtype=torch.float32, need_dw=False)
    assert torch.equal(one["dx"], got["dx"])


@pytest.mark.parametrize("n", [64, 37])
def test_fp32_gradients_nonfinite_and_extreme_dy(n):
    """An infinite dy gives infinite gradients (not NaN), NaN stays in its row and
    column, the smallest and largest dy keep their values."""
    m, k = 70, 48
    w = rand(20, n, k).abs().add(0.5).bfloat16()
    x = rand(21, m, k).abs().add(0.5).bfloat16()
    dy = rand(22, m, n)
    clean = B.linear_bwd(x, w, dy, grad_dtype=torch.float32)
    dy[5, 3] = float("inf")
    dy[9, 7] = float("nan")
    got = B.linear_bwd(x, w, dy, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool((got["dx"][5] == float("inf")).all()) and bool(torch.isnan(got["dx"][9]).all())
    assert bool((got["dw"][3] == float("inf")).all()) and bool(torch.isnan(got["dw"][7]).all())
    rows = [i for i in range(m) if i not in (5, 9)]
    cols = [i for i in range(n) if i not in (3, 7)]
    assert torch.equal(got["dx"][rows], clean["dx"][rows])
    assert torch.equal(got["dw"][cols], clean["dw"][cols])
    one = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    for v in (3.38e38, 1.2345678e-30, -7.654321e30, 0.0):
        dx = B.linear_bwd(None, one, torch.full((4, 1), v, device="cuda"), need_dw=False,
                          grad_dtype=torch.float32)["dx"].double()
        assert bool(((dx - v).abs() <= SUM2 * abs(v)).all()), v


def test_fp32_gradients_in_a_graph():
    """Captured, replayed three times over changed inputs: the eager bits."""
    x, w = rand(30, 300, 264, dtype=torch.bfloat16), rand(31, 136, 264, dtype=torch.bfloat16)
    dy, pre = rand(32, 300, 136), rand(33, 300, 136, dtype=torch.bfloat16)

    def call():
        return B.linear_bwd(x, w, dy, pre=pre, act="silu", bias=True, grad_dtype=torch.float32)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(3):
        dy.copy_(rand(40 + i, 300, 136))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        for key in want:
            assert torch.equal(out[key], want[key]), key


# --------------------------------------------------------- long column sums
def dbias_depth(m, n):
    """Additions on the longest way of a term into dbias: a lane's run of 64 rows and
    its runs (a wave takes every fourth row of a chunk), three waves, a sixteenth of
    the chunks, 16 sums."""
    span = 64 * (8 if n % 8 == 0 else 1)
    cols = -(-n // span)
    chunks = min(-(-1024 // cols), -(-m // 16))
    rows = -(-m // chunks)
    chunks = -(-m // rows)
    lane = -(-rows // 4)
    return min(lane, 64) + -(-lane // 64) + 3 + -(-chunks // 16) + 16


@pytest.mark.parametrize("m,n", [(1, 7), (33, 1025), (5003, 1536), (70001, 120), (16384, 50281),
                                 (1 << 20, 1025), (1 << 18, 2049), (1 << 18, 2048)])
def test_dbias_of_many_rows(m, n):
    """Terms of one sign and nearly one size, whose roundings add up: the sum stays
    within the additions on its way, at odd widths as at others, and no chunk of
    rows is missing."""
    assert dbias_depth(m, n) < 300
    col = torch.linspace(0.05, 0.15, n, device="cuda")
    dy = torch.empty(m, n, device="cuda")
    dy.copy_(col)
    dy[m // 3] = 1.0
    w = torch.zeros(n, 8, device="cuda")
    db = B.linear_bwd(None, w, dy, bias=True, need_dx=False, need_dw=False)["dbias"]
    torch.cuda.synchronize()
    want = (m - 1) * col.double() + 1.0
    bad = (db.double() - want).abs() / want
    log("dbias", m, n, "%.3g of the sum, bound %.3g" % (float(bad.max()), dbias_depth(m, n) * U))
    assert bool((bad <= dbias_depth(m, n) * U).all())


@pytest.mark.parametrize("m,n", [(1 << 20, 2049), (1 << 20, 2304)])
def test_dbias_past_2_31(m, n):
    """Past 2^31 elements of dy, a chunk of rows in a thousand of the sum."""
    col = torch.linspace(0.05, 0.15, n, device="cuda").bfloat16()
    dy = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    dy.copy_(col)
    w = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    db = B.linear_bwd(None, w, dy, bias=True, need_dx=False, need_dw=False)["dbias"]
    torch.cuda.synchronize()
    want = m * col.double()
    bad = (db.double() - want).abs() / want
    assert dbias_depth(m, n) * U < 1e-3 / 16
    assert bool((bad <= dbias_depth(m, n) * U).all())


def norm_depth(rows, dim):
    """Additions on the longest way of a term into dweight or dbias: a run of 64 rows of
    one of 512 blocks' groups (64 partial rows past 8192 columns) and its runs, the
    groups, a sixteenth of the partial rows, 16 sums."""
    if dim > 8192:
        parts, groups = min(rows, 64), 1
        lane = -(-rows // parts)
    else:
        waves = -(-dim // 512)
        groups = 8 // waves if waves < 8 else 1
        parts = min(-(-rows // groups), 512)
        lane = -(-rows // (parts * groups))
    return min(lane, 64) + -(-lane // 64) + groups + -(-parts // 16) + 16


@pytest.mark.parametrize("rows,dim", [(1, 9), (100, 9001), (1100, 520), (1 << 19, 4096),
                                      (1 << 20, 773), (200000, 8200), (300000, 40),
                                      (1 << 20, 2304)])
def test_norm_column_sums_of_many_rows(rows, dim):
    """Terms of one sign and nearly one size, whose roundings add up: dweight and dbias
    stay within the additions on their way, and no row is missing."""
    assert norm_depth(rows, dim) < 250
    col = torch.linspace(0.05, 0.15, dim, device="cuda")
    dy = torch.empty(rows, dim, device="cuda")
    dy.copy_(col)
    dy[rows // 3] = 1.0
    s = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    mean = torch.full((rows,), -1.0, device="cuda")
    g = B.layernorm_bwd(s, dy, mean, torch.ones(rows, device="cuda"), dx_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want = (rows - 1) * col.double() + 1.0                # xh = 1: dweight is dbias
    for key in ("dweight", "dbias"):
        bad = (g[key].double() - want).abs() / want
        log("norm", key, rows, dim, "%.3g of the sum, bound %.3g" % (
            float(bad.max()), norm_depth(rows, dim) * U))
        assert bool((bad <= norm_depth(rows, dim) * U).all()), key


# ------------------------------------- rows past 8192 columns, many to a block
def wide_norm_inputs(rows, dim, ti, tr, to, seed):
    x = rand(seed, rows, dim, dtype=DT[ti], offset=0.5)
    r = rand(seed + 1, rows, dim, dtype=DT[tr], scale=2.0, offset=-3.0)
    w, b = rand(seed + 2, dim, scale=0.3, offset=1.0), rand(seed + 3, dim)
    return x, r, w, b, rand(seed + 4, rows, dim, dtype=DT[to])


@pytest.mark.parametrize("with_dsum", [True, False])
@pytest.mark.parametrize("rows,dim,ti,tr,to", [
    (700, 8200, "bf16", "f32", "bf16"), (1100, 9001, "f32", "bf16", "bf16"),
    (1030, 16384, "bf16", "bf16", "f32"), (65, 12345, "bf16", "f32", "f32"),
    (1537, 8193, "f32", "f32", "f32"), (600, 32768, "bf16", "f32", "bf16")])
def test_norm_wide_rows(rows, dim, ti, tr, to, with_dsum):
    """More rows than the 512 blocks of the backward and the 64 partial rows of its
    column sums, at even and odd widths."""
    log("norm wide", rows, dim, ti, tr, to, with_dsum)
    x, r, w, b, dy = wide_norm_inputs(rows, dim, ti, tr, to, 50 + rows)
    got = B.layernorm_fwd(x, w, b, residual=r, eps=1e-3, out_dtype=DT[to], save_stats=True)
    y, s, mean, rstd, ty, tm, ts = ref.norm_fwd(x, r, w, b, 0.0010000000474974513)
    check(got["y"], y, ty, "y")
    check(got["sum"], s, U * s.abs(), "sum")
    check(got["mean"], mean, tm + U * mean.abs(), "mean")
    check(got["rstd"], rstd, ts, "rstd")
    del y, s, ty
    ds = r if with_dsum else None
    g = B.layernorm_bwd(x, dy, got["mean"], got["rstd"], w, dsum=ds, dx_dtype=DT[tr])
    torch.cuda.synchronize()
    dx, dw, db, tx = ref.norm_bwd(x, dy, got["mean"], got["rstd"], w, ds)[:4]
    check(g["dx"], dx, tx, "dx")
    xh = (x.double() - got["mean"].double()[:, None]) * got["rstd"].double()[:, None]
    depth = (norm_depth(rows, dim) + 4) * U       # and the roundings of a term
    check(g["dweight"], dw, depth * (dy.double() * xh).abs().sum(0), "dweight")
    check(g["dbias"], db, depth * dy.double().abs().sum(0), "dbias")
    again = B.layernorm_bwd(x, dy, got["mean"], got["rstd"], w, dsum=ds, dx_dtype=DT[tr])
    for k in g:
        assert torch.equal(g[k], again[k]), k


@pytest.mark.parametrize("dim", [8200, 9001, 32767])
def test_norm_wide_rows_in_place(dim):
    """sum over residual and dx over dsum give the same bits."""
    rows = 600
    x, r, w, _, dy = wide_norm_inputs(rows, dim, "bf16", "f32", "bf16", 90)
    want = B.layernorm_fwd(x, w, residual=r, out_dtype=torch.bfloat16, save_stats=True)
    g = B.layernorm_bwd(want["sum"], dy, want["mean"], want["rstd"], w, dsum=r)
    d = B.make_norm_desc(rows, dim)
    rr, y = r.clone(), torch.empty_like(x)
    assert B.ss_layernorm_fwd(d, x, rr, w, None, y, rr, None, None) == B.SS_OK
    assert torch.equal(rr, want["sum"]) and torch.equal(y, want["y"])
    d = B.make_norm_desc(rows, dim, in_dtype=B.SS_F32)
    nb = B.ss_layernorm_workspace_bytes(d)
    dx, dw, db = r.clone(), torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    assert B.ss_layernorm_bwd(d, want["sum"], w, want["mean"], want["rstd"], dy, dx, dx, dw, db,
                              B.workspace(nb, "cuda"), nb) == B.SS_OK
    torch.cuda.synchronize()
    assert torch.equal(dx, g["dx"])
    assert torch.equal(dw, g["dweight"]) and torch.equal(db, g["dbias"])


# --------------------------------------------------- a block in bf16, call by call
def test_mamba_block_bf16():
    """A Mamba block's calls in bf16 with its residual stream and the gradients behind
    the scan and the conv in fp32: every norm and projection of it against its 64-bit
    form on the inputs that the call in front of it gave."""
    Bt, L, dm, di, N, R, K = 2, 150, 96, 192, 16, 12, 4
    bf = torch.bfloat16
    p = lambda seed, *s, **kw: rand(seed, *s, dtype=bf, **kw)
    flat = lambda t: t.reshape(-1, t.shape[-1])
    res, dout = rand(400, Bt, L, dm), rand(401, Bt, L, dm)
    nw, nb = rand(402, dm, scale=0.2, offset=1.0), rand(403, dm, scale=0.1)
    wi = p(404, 2 * di, dm, scale=dm ** -0.5)
    cw, cb = rand(405, di, K, scale=0.5), rand(406, di, scale=0.1)
    wx, wt = p(407, R + 2 * N, di, scale=di ** -0.5), p(408, di, R, scale=0.3)
    wo = p(409, dm, di, scale=di ** -0.5)
    A, D, tb = -torch.exp(0.5 * rand(410, di, N)), rand(411, di), rand(412, di, offset=-1.0)

    def fwd(x, w, residual=None, out_dtype=None):
        y = B.linear_fwd(x, w, residual=residual, out_dtype=out_dtype)
        want, _, tol, _ = ref.linear_fwd(flat(x), w, None,
                                         None if residual is None else flat(residual), "none")
        check(flat(y), want, tol, "forward %s" % (tuple(w.shape),))
        return y

    def bwd(x, w, dy, gt):
        g = B.linear_bwd(x, w, dy, bias=True, grad_dtype=gt)
        x, dy = flat(x), flat(dy)
        if gt == torch.float32:
            dx, dw, tx, tw = bwd_fp32(x, w, dy, None, "none")
        else:
            dx, dw, _, tx, tw, _ = ref.linear_bwd(x, w, dy, None, "none")
        check(flat(g["dx"]), dx, tx, "dx %s" % (tuple(w.shape),))
        check(g["dw"], dw, tw, "dw %s" % (tuple(w.shape),))
        d = dy.double()
        check(g["dbias"], d.sum(0), dbias_depth(*d.shape) * U * d.abs().sum(0), "dbias")
        return g

    n = B.layernorm_fwd(res, nw, nb, out_dtype=bf, save_stats=True)
    y, _, mean, rstd, ty, tm, ts = ref.norm_fwd(flat(res), None, nw, nb, 9.999999747378752e-06)
    check(flat(n["y"]), y, ty, "norm")
    check(n["mean"].view(-1), mean, tm + U * mean.abs(), "mean")
    check(n["rstd"].view(-1), rstd, ts, "rstd")
    xz = fwd(n["y"], wi)
    xu, z = xz[..., :di].contiguous(), xz[..., di:].contiguous()
    u = B.conv1d_fwd(xu, cw, cb)
    xdb = fwd(u, wx)
    Bm, Cm = xdb[..., R:R + N], xdb[..., R + N:]
    delta = fwd(xdb[..., :R], wt)
    y = B.scan_fwd(u, delta, A, Bm, Cm, D=D, delta_bias=tb, z=z, out_dtype=bf)
    out = fwd(y, wo, residual=res, out_dtype=torch.float32)
    assert out.dtype == torch.float32 and bool(torch.isfinite(out).all())

    go = bwd(y, wo, dout, bf)
    gs = B.scan_bwd(u, delta, A, Bm, Cm, go["dx"], D=D, delta_bias=tb, z=z)
    f32 = torch.float32
    gt = bwd(xdb[..., :R], wt, gs["ddelta"], f32)
    gx = bwd(u, wx, torch.cat([gt["dx"], gs["dB"], gs["dC"]], dim=-1), f32)
    gc = B.conv1d_bwd(xu, cw, gs["du"] + gx["dx"], cb)
    gi = bwd(n["y"], wi, torch.cat([gc["dx"], gs["dz"]], dim=-1), f32)
    gn = B.layernorm_bwd(res, gi["dx"], n["mean"], n["rstd"], nw, dsum=dout)
    torch.cuda.synchronize()
    dx, dw, db, tx = ref.norm_bwd(flat(res), flat(gi["dx"]), n["mean"].view(-1),
                                  n["rstd"].view(-1), nw, flat(dout))[:4]
    check(flat(gn["dx"]), dx, tx, "norm dx")
    d = flat(gi["dx"]).double()
    xh = (flat(res).double() - n["mean"].double().view(-1, 1)) * n["rstd"].double().view(-1, 1)
    depth = (norm_depth(Bt * L, dm) + 4) * U
    check(gn["dweight"], dw, depth * (d * xh).abs().sum(0), "norm dweight")
    check(gn["dbias"], db, depth * d.abs().sum(0), "norm dbias")
