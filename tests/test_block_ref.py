"""The 64-bit forms that the GPU tests of the operators around the scan compare with,
themselves against differences and definitions (CPU)."""
import math

import pytest
import torch

import block_ref as ref


def central(loss, t, grad, h=1e-6):
    """grad against central differences of loss over every element of t."""
    flat, g = t.view(-1), grad.reshape(-1)
    assert flat.numel() == g.numel()
    for i in range(flat.numel()):
        old = float(flat[i])
        flat[i] = old + h
        up = loss()
        flat[i] = old - h
        down = loss()
        flat[i] = old
        assert abs((up - down) / (2 * h) - float(g[i])) < 1e-7


@pytest.mark.parametrize("name", ["silu", "gelu", "softplus", "none"])
def test_linear_bwd_against_differences(name, monkeypatch):
    """ref.linear_bwd's own gradients, each activation, for a loss of ref.linear_fwd."""
    # operands in float64: what the tolerances count as their rounding
    monkeypatch.setitem(ref.HALF, torch.float64, 2.0 ** -53)
    g = torch.Generator().manual_seed(11)
    x, w, dy, r = (torch.randn(s, generator=g, dtype=torch.float64)
                   for s in ((5, 4), (3, 4), (5, 3), (5, 3)))
    b = torch.randn(3, generator=g, dtype=torch.float64)

    def loss():
        return float((ref.linear_fwd(x, w, b, r, name)[0] * dy).sum())
    pre = ref.linear_fwd(x, w, b, r, name)[1]
    dx, dw, db = ref.linear_bwd(x, w, dy, None if name == "none" else pre, name)[:3]
    for t, grad in ((x, dx), (w, dw), (b, db)):
        central(loss, t, grad)


@pytest.mark.parametrize("name", ["silu", "gelu", "softplus"])
def test_activations_from_their_definitions(name):
    """A relative error d of erfc's argument x = -v / sqrt(2) becomes 2 x^2 d = v^2 d of
    its value (erfc' / erfc -> -2 x), and either side's x carries two roundings of 2^-53:
    v^2 2^-51 beside the 1e-14 that the rest gets."""
    for v in (-30.0, -5.0, -1.0, -0.1, 0.0, 0.3, 2.0, 7.5, 40.0):
        want = {"silu": v / (1 + math.exp(-v)), "gelu": v * 0.5 * math.erfc(-v / math.sqrt(2)),
                "softplus": math.log1p(math.exp(-abs(v))) + max(v, 0.0)}[name]
        got = float(ref.act(name, torch.tensor(v, dtype=torch.float64)))
        lim = 1e-14 + (v * v * 2.0 ** -51 if name == "gelu" else 0.0)
        assert abs(got - want) <= lim * max(abs(want), 1e-300), v
