"""CPU-side checks of a gated recurrent block's operators: descriptors match the headers,
invalid arguments are refused before any HIP call, the binding refuses what the library
would read wrongly, and the 64-bit forms' gradients against autograd and differences."""
import os
import re
import subprocess
import ctypes

import pytest
import torch

from selective_state_space_69_amd import binding as B
import gated_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 20          # an aligned non-null "device pointer"; never dereferenced
INV, UNS, WSP = B.SS_ERR_INVALID_ARG, B.SS_ERR_UNSUPPORTED, B.SS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from selective_state_space_69_amd import build
        build.build(verbose=False)
    return B.load_library()


def at(i):
    return F + (i << 24)


def rec_desc(**kw):
    return B.make_rec_desc(**{**dict(batch=2, seqlen=4096, dim=64), **kw})


def rec_fwd(d, **kw):
    a = {**dict(x=at(0), r=at(1), i=at(2), lam=at(3), z=None, h0=None, starts=None, lengths=None,
                y=at(4), h_last=at(5), states=at(6), workspace=at(7), ws_bytes=1 << 40), **kw}
    return B.ss_rec_fwd(d, *a.values(), stream=0)


def rec_bwd(d, **kw):
    a = {**dict(x=at(0), r=at(1), i=at(2), lam=at(3), z=None, starts=None, lengths=None,
                states=at(4), dy=at(5), dh_last=None, dx=at(6), dr=at(7), di=at(8), dz=None,
                dlam=at(9), dh0=at(10), workspace=at(11), ws_bytes=1 << 40), **kw}
    return B.ss_rec_bwd(d, *a.values(), stream=0)


def rec_step(d, **kw):
    a = {**dict(h=at(0), x=at(1), r=at(2), i=at(3), lam=at(4), z=None, y=at(5)), **kw}
    return B.ss_rec_step(d, *a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INV), (dict(seqlen=0), INV), (dict(seqlen=1 << 31), INV), (dict(dim=0), INV),
    (dict(dim=(1 << 20) + 1), INV), (dict(batch=(1 << 22) + 1), INV),
    (dict(batch=1 << 21, dim=129), INV), (dict(batch=1 << 15, seqlen=1 << 20), INV),
    (dict(x_stride=63), INV), (dict(r_stride=63), INV), (dict(i_stride=(1 << 20) + 1), INV),
    (dict(z_stride=-1), INV), (dict(in_dtype=2), UNS), (dict(out_dtype=-1), UNS),
    (dict(decay=0.0), INV), (dict(decay=-1.0), INV), (dict(decay=float("inf")), INV),
    (dict(decay=float("nan")), INV),
])
def test_rec_descriptor(kw, code):
    d = rec_desc(**kw)
    assert rec_fwd(d) == code and rec_bwd(d) == code
    for op in (B.SS_REC_FWD, B.SS_REC_BWD):
        assert B.ss_rec_workspace_bytes(d, op) == 0
    if "seqlen" not in kw:
        d.seqlen = 1
        if kw != dict(batch=1 << 15, seqlen=1 << 20):
            assert rec_step(d) == code
    d = rec_desc()
    d.reserved = 1
    assert rec_fwd(d) == INV
    assert B.ss_rec_workspace_bytes(rec_desc(), 2) == 0


def test_rec_grid():
    # workgroups of 512 threads and 32 channels: their threads have to stay below 2^32
    for batch, dim in (((1 << 21) + 1, 64), ((1 << 20) + 1, 65), ((1 << 21) // 3 + 1, 150)):
        assert rec_fwd(rec_desc(batch=batch, dim=dim)) == INV
        assert B.ss_rec_workspace_bytes(rec_desc(batch=batch, dim=dim), B.SS_REC_BWD) == 0
    for batch, dim in ((1 << 21, 64), (1 << 20, 65), ((1 << 21) // 3, 150)):
        assert B.ss_rec_workspace_bytes(rec_desc(batch=batch, dim=dim), B.SS_REC_BWD) > 0


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(r=None), INV), (dict(i=None), INV), (dict(lam=None), INV),
    (dict(y=None), INV), (dict(y=at(0)), INV), (dict(h_last=at(4)), INV), (dict(states=at(5)), INV),
    (dict(y=at(8), h0=at(8)), INV), (dict(states=at(8), h0=at(8)), INV), (dict(h_last=at(3)), INV),
    (dict(starts=at(8), states=at(8)), INV), (dict(lengths=at(8), y=at(8)), INV),
    (dict(x=at(0) + 2), INV), (dict(z=at(8) + 8), INV), (dict(lam=at(3) + 4), INV),
    (dict(h0=at(8) + 4), INV), (dict(y=at(4) + 2), INV), (dict(lengths=at(8) + 4), INV),
    (dict(workspace=None), WSP), (dict(ws_bytes=64), WSP), (dict(workspace=at(7) + 16), WSP),
])
def test_rec_fwd_arguments(kw, code):
    assert rec_fwd(rec_desc(), **kw) == code


def test_rec_strides_relax_alignment():
    """A tensor with a row stride needs its element alignment only."""
    d = rec_desc(x_stride=80)
    assert rec_fwd(d, x=at(0) + 1) == INV
    assert rec_fwd(d, x=at(0) + 2, y=None) == INV      # aligned enough: refused for y alone
    assert rec_fwd(d, x=at(0) + 2, workspace=None) == WSP


@pytest.mark.parametrize("kw,code", [
    (dict(states=None), INV), (dict(dy=None), INV), (dict(dx=None), INV), (dict(dr=None), INV),
    (dict(di=None), INV), (dict(dlam=None), INV), (dict(z=at(12)), INV), (dict(dz=at(12)), INV),
    (dict(dx=at(0)), INV), (dict(dr=at(6)), INV), (dict(di=at(5)), INV), (dict(dlam=at(3)), INV),
    (dict(dh0=at(4)), INV), (dict(dh0=at(12), dh_last=at(12)), INV), (dict(z=at(12), dz=at(12)), INV),
    (dict(dy=at(5) + 2), INV), (dict(states=at(4) + 4), INV), (dict(dlam=at(9) + 4), INV),
    (dict(workspace=None), WSP), (dict(ws_bytes=64), WSP),
])
def test_rec_bwd_arguments(kw, code):
    assert rec_bwd(rec_desc(), **kw) == code


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(x=None), dict(lam=None), dict(y=None), dict(y=at(0)), dict(y=at(2)),
    dict(h=at(1)), dict(h=at(0) + 4), dict(y=at(5) + 4), dict(z=at(5)),
])
def test_rec_step_arguments(kw):
    assert rec_step(rec_desc(seqlen=1), **kw) == INV
    assert rec_step(rec_desc(seqlen=2)) == INV


def test_rec_workspace_follows_the_plan():
    """None where the channels fill the GPU; chunks' carries where they do not."""
    assert B.ss_rec_workspace_bytes(rec_desc(batch=8, seqlen=2048, dim=2560), B.SS_REC_FWD) == 0
    n = B.ss_rec_workspace_bytes(rec_desc(batch=1, seqlen=1 << 20, dim=64), B.SS_REC_FWD)
    assert 0 < n < 1 << 20
    assert B.ss_rec_workspace_bytes(rec_desc(batch=1, seqlen=1 << 20, dim=64), B.SS_REC_BWD) > n


def test_descriptors_match_the_headers(tmp_path):
    structs = [("ss_rec_desc_t", B.ss_rec_desc_t), ("ss_glu_desc_t", B.ss_glu_desc_t),
               ("ss_q8_pack_desc_t", B.ss_q8_pack_desc_t), ("ss_q8_desc_t", B.ss_q8_desc_t)]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "ss_rec.h"', '#include "ss_glu.h"',
           '#include "ss_q8.h"', "int main(void) {"]
    want = []
    for name, t in structs:
        src.append('printf("%%zu\\n", sizeof(%s));' % name)
        want.append(ctypes.sizeof(t))
        for f, _ in t._fields_:
            src.append('printf("%%zu\\n", offsetof(%s, %s));' % (name, f))
            want.append(getattr(t, f).offset)
    c = tmp_path / "d.c"
    c.write_text("\n".join(src + ["return 0; }"]))
    exe = str(tmp_path / "d")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == want


def test_headers_name_every_constant():
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in ("ss_rec.h", "ss_glu.h"))
    for name in ("SS_REC_CHUNK", "SS_REC_FWD", "SS_REC_BWD", "SS_GLU_FWD", "SS_GLU_BWD"):
        m = re.search(r"#define %s (\d+)" % name, text)
        assert m and int(m.group(1)) == getattr(B, name)
    assert ref.CHUNK == B.SS_REC_CHUNK


def test_binding_refuses():
    x = torch.zeros(2, 3, 8)
    lam = torch.zeros(8)
    with pytest.raises(ValueError, match="on the GPU"):
        B.rec_fwd(x, x, x, lam)
    call = B._rec_fwd

    def fwd(**kw):
        a = {**dict(raw=0, x=x, r=x, i=x, lam=lam, z=None, h0=None, starts=None, lengths=None,
                    decay=8.0, odt=torch.float32, return_last=False, save_states=False), **kw}
        return call(*a.values())
    for kw, what in [
        (dict(x=torch.zeros(2, 8)), "batch, seqlen"), (dict(r=torch.zeros(2, 3, 7)), "r must have shape"),
        (dict(i=x.bfloat16()), "one dtype"), (dict(z=torch.zeros(2, 4, 8)), "z must have shape"),
        (dict(x=x.double(), r=x.double(), i=x.double()), "float32 or bfloat16"),
        (dict(lam=lam.bfloat16()), "lam must be float32"), (dict(lam=torch.zeros(7)), "lam must have shape"),
        (dict(h0=torch.zeros(2, 7)), "h0 must have shape"), (dict(h0=torch.zeros(2, 16)[:, ::2]), "contiguous"),
        (dict(starts=torch.zeros(2, 3)), "starts must be"), (dict(starts=torch.zeros(2, 4, dtype=torch.uint8)), "shape"),
        (dict(lengths=torch.zeros(2)), "lengths must be int32"),
        (dict(lengths=torch.zeros(3, dtype=torch.int32)), "shape"),
        (dict(odt=torch.float16), "float32 or bfloat16"),
        (dict(x=torch.zeros(1, 3, 8).expand(2, 3, 8)), "evenly|overlap"),
    ]:
        with pytest.raises(ValueError, match=what):
            fwd(**kw)
    with pytest.raises(ValueError, match="batch, dim"):
        B._rec_step(0, torch.zeros(2, 8), x, x, x, lam, None, 8.0, torch.float32)


# ------------------------------------------------ gated feed-forward half
def glu_desc(**kw):
    return B.make_glu_desc(**{**dict(rows=64, in_dim=64, out_dim=64), **kw})


def glu_fwd(d, **kw):
    a = {**dict(x=at(0), w=at(1), bias=None, y=at(2), pre=None, workspace=at(3), ws_bytes=1 << 40), **kw}
    return B.ss_glu_fwd(d, *a.values(), stream=0)


def glu_bwd(d, **kw):
    a = {**dict(x=at(0), w=at(1), pre=at(2), dy=at(3), dx=at(4), dw=at(5), dbias=None, workspace=at(6),
                ws_bytes=1 << 40), **kw}
    return B.ss_glu_bwd(d, *a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=(1 << 28) + 1), INV), (dict(in_dim=0), INV),
    (dict(in_dim=(1 << 20) + 1), INV), (dict(out_dim=0), INV), (dict(out_dim=(1 << 19) + 1), INV),
    (dict(rows=1 << 28, in_dim=256), INV), (dict(rows=1 << 28, out_dim=65), INV),
    (dict(in_dim=1 << 20, out_dim=1 << 15), INV), (dict(x_stride=63), INV),
    (dict(x_stride=(1 << 20) + 1), INV), (dict(in_dtype=2), UNS), (dict(out_dtype=-1), UNS),
    (dict(act=B.SS_ACT_SOFTPLUS), UNS), (dict(act=-1), UNS),
])
def test_glu_descriptor(kw, code):
    if kw == dict(in_dim=1 << 20, out_dim=1 << 15):       # w of 2^36 elements
        kw = {**kw, "rows": 1}
    d = glu_desc(**kw)
    assert glu_fwd(d) == code and glu_bwd(d) == code
    for op in (0, 1):
        assert B.ss_glu_workspace_bytes(d, op) == 0
    assert B.ss_glu_workspace_bytes(glu_desc(), 2) == 0
    assert glu_bwd(glu_desc(grad_dtype=5)) == UNS
    assert glu_fwd(glu_desc(grad_dtype=5), y=None) == INV        # not read by the forward


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(y=at(0)), INV),
    (dict(y=at(4), pre=at(4)), INV), (dict(pre=at(1)), INV), (dict(bias=at(2)), INV),
    (dict(x=at(0) + 2), INV), (dict(w=at(1) + 8), INV), (dict(pre=at(5) + 2), INV),
])
def test_glu_fwd_arguments(kw, code):
    assert glu_fwd(glu_desc(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), INV), (dict(pre=None), INV), (dict(dy=None), INV), (dict(x=None), INV),
    (dict(dx=None, dw=None), INV), (dict(dx=at(3)), INV), (dict(dw=at(0)), INV), (dict(dx=at(5)), INV),
    (dict(dbias=at(2)), INV), (dict(dy=at(3) + 2), INV), (dict(dw=at(5) + 8), INV),
    (dict(workspace=None), WSP), (dict(ws_bytes=64), WSP), (dict(workspace=at(6) + 16), WSP),
])
def test_glu_bwd_arguments(kw, code):
    assert glu_bwd(glu_desc(), **kw) == code


def test_glu_workspace():
    """d of both halves, doubled where one bf16 per value cannot hold it; none to decode."""
    assert B.ss_glu_workspace_bytes(glu_desc(rows=8), B.SS_GLU_FWD) == 0
    one = B.ss_glu_workspace_bytes(glu_desc(rows=512), B.SS_GLU_BWD)
    two = B.ss_glu_workspace_bytes(glu_desc(rows=512, grad_dtype=B.SS_F32), B.SS_GLU_BWD)
    assert one >= 512 * 128 * 2 and two >= one + 512 * 128 * 2


# ------------------------------------------------ 8-bit integers
def q8_linear(d, **kw):
    a = {**dict(xq=at(0), xs=at(1), wq=at(2), ws=at(3), bias=None, residual=None, y=at(4), workspace=at(5),
                ws_bytes=1 << 40), **kw}
    return B.ss_q8_linear(d, *a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=1 << 31), INV), (dict(dim=0), INV), (dict(dim=(1 << 20) + 1), INV),
    (dict(x_stride=63), INV), (dict(q_stride=63), INV), (dict(q_stride=(1 << 20) + 1), INV), (dict(dtype=2), UNS),
])
def test_q8_pack_descriptor(kw, code):
    d = B.make_q8_pack_desc(**{**dict(rows=4, dim=64), **kw})
    assert B.ss_q8_pack(d, at(0), at(1), at(2), stream=0) == code


def test_q8_pack_arguments():
    d = B.make_q8_pack_desc(4, 64)
    for a in ((None, at(1), at(2)), (at(0), None, at(2)), (at(0), at(1), None), (at(0), at(0), at(2)),
              (at(0), at(1), at(1)), (at(0), at(1), at(0)), (at(0) + 2, at(1), at(2)), (at(0), at(1) + 8, at(2)),
              (at(0), at(1), at(2) + 4)):
        assert B.ss_q8_pack(d, *a, stream=0) == INV
    d.reserved = 1
    assert B.ss_q8_pack(d, at(0), at(1), at(2), stream=0) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=(1 << 28) + 1), INV), (dict(in_dim=0), INV), (dict(in_dim=(1 << 16) + 1), INV),
    (dict(out_dim=0), INV), (dict(out_dim=(1 << 20) + 1), INV), (dict(rows=1 << 28, in_dim=129), INV),
    (dict(rows=1 << 28, out_dim=129), INV), (dict(x_stride=63), INV), (dict(w_stride=63), INV),
    (dict(w_stride=(1 << 20) + 1), INV), (dict(out_dtype=2), UNS), (dict(res_dtype=7), UNS), (dict(act=4), UNS),
])
def test_q8_descriptor(kw, code):
    d = B.make_q8_desc(**{**dict(rows=64, in_dim=64, out_dim=64), **kw})
    assert q8_linear(d) == code
    assert B.ss_q8_workspace_bytes(d) == 0
    d.reserved = 1
    assert q8_linear(d) != B.SS_OK


@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), INV), (dict(xs=None), INV), (dict(wq=None), INV), (dict(ws=None), INV), (dict(y=None), INV),
    (dict(y=at(0)), INV), (dict(y=at(3)), INV), (dict(bias=at(4)), INV), (dict(xq=at(0) + 8), INV),
    (dict(wq=at(2) + 1), INV), (dict(xs=at(1) + 4), INV), (dict(residual=at(6) + 2), INV),
    (dict(workspace=None), WSP), (dict(ws_bytes=64), WSP),
])
def test_q8_arguments(kw, code):
    assert q8_linear(B.make_q8_desc(64, 63, 64), **kw) == code
    if code == INV:
        d = B.make_q8_desc(64, 63, 64, out_dtype=B.SS_F32, res_dtype=B.SS_BF16)
        assert q8_linear(d, residual=at(4)) == INV         # in place only in one type


def test_more_binding_refusals():
    x, w = torch.zeros(3, 8), torch.zeros(10, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        B.glu_fwd(x, w)
    with pytest.raises(KeyError):
        B.glu_fwd(x, w, act="softplus")
    fwd = B._glu_fwd
    for a, what in [((x, torch.zeros(9, 8), None), "rows"), ((torch.zeros(3, 7), w, None), "columns"),
                    ((x.bfloat16(), w, None), "one dtype"), ((x, w, torch.zeros(5)), "bias must have shape"),
                    ((x, w, torch.zeros(10).bfloat16()), "bias must be float32")]:
        with pytest.raises(ValueError, match=what):
            fwd(0, *a, B.SS_ACT_SILU, torch.float32, False)
    pre, dy = torch.zeros(3, 10), torch.zeros(3, 5)
    for a, what in [((None, w, dy, pre), "dw needs x"), ((x, w, torch.zeros(3, 4), pre), "dy must have shape"),
                    ((x, w, dy, pre[:, :8]), "pre must have shape"), ((x, w, dy, pre.bfloat16()), "w's dtype"),
                    ((x[:2], w, dy, pre), "x must have shape"), ((x.bfloat16(), w, dy, pre), "one dtype")]:
        with pytest.raises(ValueError, match=what):
            B._glu_bwd(0, *a, B.SS_ACT_SILU, False, torch.float32, True, True)
    q, s = torch.zeros(3, 8, dtype=torch.int8), torch.zeros(3)
    wq, ws = torch.zeros(5, 8, dtype=torch.int8), torch.zeros(5)
    with pytest.raises(ValueError, match="on the GPU"):
        B.q8_linear((q, s), (wq, ws))
    for a, what in [((q[:, :7], s, wq, ws), "columns"), ((q.float(), s, wq, ws), "int8"),
                    ((q, s.bfloat16(), wq, ws), "float32"), ((q, s[:2], wq, ws), "x's scales must have shape"),
                    ((q, s, wq, ws[:4]), "w's scales must have shape")]:
        with pytest.raises(ValueError, match=what):
            B._q8_linear(0, *a, None, None, 0, torch.float32)
    with pytest.raises(ValueError, match="residual must have shape"):
        B._q8_linear(0, q, s, wq, ws, None, torch.zeros(3, 4), 0, torch.float32)


# ------------------------------------------------ the 64-bit forms
def test_reference_glu_gradients():
    g = torch.Generator().manual_seed(3)
    x, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4), (6, 4), (5, 3)))
    b = torch.randn(6, generator=g, dtype=torch.float64)
    for name in ("silu", "gelu", "none"):
        def loss():
            return float((ref.glu_fwd(x, w, b, name)[0] * dy).sum())
        pre = x @ w.t() + b
        grads = ref.glu_bwd(x, w, dy, pre, name, torch.float64)[:3]
        for t, grad in zip((x, w, b), grads):
            for i in range(t.numel()):
                old = float(t.view(-1)[i])
                t.view(-1)[i] = old + 1e-6
                up = loss()
                t.view(-1)[i] = old - 1e-6
                dn = loss()
                t.view(-1)[i] = old
                assert abs((up - dn) / 2e-6 - float(grad.reshape(-1)[i])) < 1e-7


def test_reference_q8_is_its_definition():
    """Against whole-number arithmetic without rounding."""
    from fractions import Fraction
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 50, generator=g)
    x[0] = torch.arange(50) * 0.5                  # many ties: 127 x / 24.5 in halves
    x[0, 49] = 63.5
    x[1] = 0.0
    x[2, 7] = float("inf")
    q, s = ref.q8_pack(x)
    assert not bool(q[1:3].any()) and float(s[1]) == 0.0 and bool(torch.isnan(s[2]))
    for row in (0, 3, 4, 5):
        top = max(abs(Fraction(float(v))) for v in x[row])
        for c in range(50):
            assert int(q[row, c]) == round(127 * Fraction(float(x[row, c])) / top)     # ties to even


def _rec_inputs(b=2, l=9, d=3):
    g = torch.Generator().manual_seed(7)

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)
    t = {"x": rand(b, l, d), "r": rand(b, l, d), "i": rand(b, l, d), "lam": rand(d), "z": rand(b, l, d),
         "h0": rand(b, d)}
    m = {"starts": torch.rand(b, l, generator=g) < 0.2, "lengths": torch.tensor([l, 5])}
    return t, m, rand(b, l, d), rand(b, d)


def test_reference_recurrence_is_its_definition():
    t, m, _, _ = _rec_inputs()
    y, last, states, *_ = ref.Rec(**t, **m).fwd()
    for b in range(2):
        h = t["h0"][b]
        for k in range(9):
            if k < int(m["lengths"][b]):
                a = torch.exp(-8 * ref.softplus(t["lam"]) * torch.sigmoid(t["r"][b, k]))
                h = (0 if m["starts"][b, k] else a * h) + (1 - a * a).sqrt() * torch.sigmoid(t["i"][b, k]) * t["x"][b, k]
                want = h * t["z"][b, k] * torch.sigmoid(t["z"][b, k])
            else:
                want = torch.zeros(3, dtype=torch.float64)
            assert torch.allclose(y[b, k], want, rtol=1e-12, atol=1e-14)
        assert torch.allclose(last[b], h, rtol=1e-12, atol=1e-14)
    assert torch.equal(states[:, 0], t["h0"])


def test_reference_recurrence_gradients():
    t, m, dy, dh = _rec_inputs()

    def loss(t):
        y, last, *_ = ref.Rec(**t, **m).fwd()
        return (y * dy).sum() + (last * dh).sum()
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    loss(leaves).backward()
    grad, _ = ref.Rec(**t, **m).bwd(dy, dh)
    for k, v in leaves.items():
        assert torch.allclose(grad["d" + k], v.grad, rtol=1e-10, atol=1e-13), k
        step = 1e-6
        for n in range(v.numel()):
            up, dn = (({**t, k: t[k].clone()}) for _ in range(2))
            up[k].view(-1)[n] += step
            dn[k].view(-1)[n] -= step
            diff = float(loss(up) - loss(dn)) / (2 * step)
            assert abs(diff - float(grad["d" + k].reshape(-1)[n])) < 1e-7, k
