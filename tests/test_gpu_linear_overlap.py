"""Buffers of the linear layer that share memory: refused before anything is launched, but for y over the residual."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
M = N = K = 48


def _t():
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w, r, z, dy = (torch.randn(48, 48, device="cuda", generator=g).to(BF16) for _ in range(5))
    return x, w, r, z, dy


@pytest.mark.parametrize("rows", [4, 48])
def test_forward(rows):
    import cnn_convolution_implicit_gb300 as cg
    x, w, r, z, _ = _t()
    x, r, z = x[:rows], r[:rows], z[:rows]
    plan = cg.LinearPlan(rows, N, K, "silu")
    bias = torch.zeros(4 * 48 * 48, device="cuda")
    want = plan.forward(x, w, None, r)
    for bad in (dict(y=x), dict(y=x, residual=x), dict(z=x), dict(z=r, residual=r), dict(y=z, z=z), dict(y=w[:rows]), dict(z=w[48 - rows:]),
                dict(bias=bias[:48], y=bias.view(BF16)[:rows * 48].view(rows, 48)), dict(bias=bias[:48], z=bias.view(BF16)[:rows * 48].view(rows, 48))):
        kept = [t.clone() for t in (x, w, r, z)]
        with pytest.raises(cg.ConvError):
            plan.forward(**dict(dict(x=x, w=w), **bad))
        assert all(torch.equal(p, q) for p, q in zip(kept, (x, w, r, z)))
    long = torch.zeros((rows + 1) * 48, device="cuda", dtype=BF16)
    with pytest.raises(cg.ConvError):  # a part of the residual
        plan.forward(x, w, None, long[:-48].view(rows, 48), y=long[48:].view(rows, 48))
    over = r.clone()
    assert torch.equal(plan.forward(x, w, None, over, y=over), want) and torch.equal(over, want)
    pair = torch.cat([r.reshape(-1), torch.zeros(rows * 48, device="cuda", dtype=BF16)])  # next to each other is not shared
    assert torch.equal(plan.forward(x, w, None, pair[:rows * 48].view(rows, 48), y=pair[rows * 48:].view(rows, 48)), want)
    assert torch.equal(plan.forward(x, x if rows == 48 else w), plan.forward(x, x.clone() if rows == 48 else w))  # inputs may be one tensor


def test_backward():
    import cnn_convolution_implicit_gb300 as cg
    x, w, _, z, dy = _t()
    for act, zz in (("none", None), ("silu", z)):
        plan = cg.LinearPlan(M, N, K, act)
        want = plan.backward(dy, x, w, zz)
        bias = torch.zeros(4 * 48 * 48, device="cuda")
        cases = [dict(dx=dy), dict(dw=dy), dict(dx=x), dict(dw=w), dict(dx=w), dict(dw=x), dict(dbias=dy.view(torch.float32).view(-1)[:48]),
                 dict(dx=bias.view(BF16)[:48 * 48].view(48, 48), dbias=bias[:48]), dict(dx=bias.view(BF16)[:48 * 48].view(48, 48), dw=bias.view(BF16)[:48 * 48].view(48, 48))]
        if zz is not None:
            cases += [dict(dx=z), dict(dw=z)]
        for bad in cases:
            with pytest.raises(cg.ConvError):
                plan.backward(dy, x, w, zz, **bad)
        again = plan.backward(dy, x, w, zz)
        assert all(torch.equal(p, q) for p, q in zip(want, again))
        same = plan.backward(dy, dy, dy, zz)  # inputs may be one tensor
        apart = plan.backward(dy, dy.clone(), dy.clone(), zz)
        assert all(torch.equal(p, q) for p, q in zip(same, apart))
