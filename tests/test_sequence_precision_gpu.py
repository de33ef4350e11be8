"""Sigmoid, SiLU, softplus and their derivatives in the sequence operators'
fp32 plans, alone: inputs that make every other factor 1 and every other term
0, so that an output is the function's own value.

Bounds, relative, in units u = 2^-24, are those of an elementary fp32
evaluation: an exponential within 2.6 u (expf over the ranges below, measured
over 2^20 points in each), every sum, product and reciprocal within u, log(1 + e)
of e within 2 u; none of the functions' slopes in e = exp(-x) makes an error
relatively larger:
 - sigmoid = 1 / (1 + e): 2.6 + 1 + 1 u, tested with 5;
 - SiLU: one product more, tested with 6;
 - softplus = max(x, 0) + log(1 + exp(-|x|)): 2.6 + 2 u, tested with 5;
 - sigmoid' = s (1 - s), at x <= 0, where 1 - s is within u: 4.6 + 1 u and a product, tested with 8;
 - SiLU' = s + x s (1 - s): at x <= 0 that and two roundings, at x > 0 (with 1 - s as e s) 3.3 u of s and 9.9 u of the
   second term, at most 0.22 of the whole there, and one rounding; tested with 8 of the terms' magnitudes.
(The kernels' exponential and reciprocal alone are off by up to 3.3 and 1.6 u, their sigmoid by up to 4.4.)
An exponent rounded to fp32 alone, e = 2^(x log2 e), would be off by up to |x| u.
"""
import pytest
import torch

import conv2d_backward_implicit_dgrad_gb300 as dg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RANGES = [(-30.0, -16.0), (-16.0, -7.0), (-7.0, -2.0), (-2.0, 0.0), (0.0, 3.0), (3.0, 20.0)]


def points(lo, hi, *shape):
    gen = torch.Generator().manual_seed(int(7 - 3 * lo))
    return (torch.rand(shape, generator=gen, dtype=torch.float64) * (hi - lo) + lo).float().cuda()


def within(got, want, units, scale=None, name=""):
    assert got.dtype == torch.float32
    off = (got.double() - want).abs() / (U * (want.abs() if scale is None else scale))
    assert torch.isfinite(off).all() and float(off.max()) <= units, f"{name}: {float(off.max()):.3g} u"


def sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x.double()))


def softplus(x):
    x = x.double()
    return x.clamp(min=0.0) + torch.log1p(torch.exp(-x.abs()))


@pytest.mark.parametrize("d", [256, 37])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_conv_silu(lo, hi, d):
    x = points(lo, hi, 2, 300, d)
    w = torch.tensor([0.0, 1.0], device="cuda").repeat(d, 1)
    s, xd = sigmoid(x), x.double()
    with dg.CausalConvPlan(2, 300, d, 2, dtype="fp32") as plan:
        within(plan.run(x, w), xd * s, 6, name="run")
        g = plan.backward(torch.ones_like(x), x, w)
        within(g.x, s + xd * s * (1.0 - s), 8, s + xd.abs() * s * (1.0 - s), "backward")
        cache = torch.zeros(2, 1, d, device="cuda")
        within(plan.step(x[:, 5], w, cache), (xd * s)[:, 5], 6, name="step")


def scan_of(dt, **given):
    """out of a scan whose decays are 1, with B = C = u = 1 unless given."""
    b, t, d = dt.shape
    one = torch.ones(b, t, 1, 1, device="cuda")
    A = torch.zeros(d, 1, device="cuda")
    return torch.ones_like(dt), dt, A, given.get("B", one), given.get("C", one)


@pytest.mark.parametrize("d", [256, 37])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_scan_softplus(lo, hi, d):
    """One token from a state of 0: out is delta; grad_dt is then its slope, sigmoid(dt)."""
    b = 300
    dt = points(lo, hi, b, 1, d)
    args = scan_of(dt)
    with dg.ScanPlan(b, 1, d, 1, dtype="fp32") as plan:
        ck = plan.checkpoints()
        within(plan.run(*args, checkpoints=ck), softplus(dt), 5, name="run")
        g = plan.backward(torch.ones_like(dt), *args, ck)
        within(g.dt, sigmoid(dt), 5, name="grad_dt")
        cache = torch.zeros(b, d, 1, device="cuda")
        u, t, A, B, C = args
        within(plan.step(u[:, 0], t[:, 0], A, B[:, 0], C[:, 0], cache), softplus(dt)[:, 0], 5, name="step")


@pytest.mark.parametrize("d", [256, 37])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_scan_softplus_handed_through_chunks(lo, hi, d):
    """A long row, cut into chunks: the first token's delta is the state, which tokens with a delta of 0 (dt of minus
    infinity) hand on as it is."""
    t = 600
    dt = points(lo, hi, 1, t, d)
    dt[:, 1:] = float("-inf")
    with dg.ScanPlan(1, t, d, 1, dtype="fp32") as plan:
        final = torch.empty(1, d, 1, device="cuda")
        plan.run(*scan_of(dt), final_state=final)
    within(final[..., 0], softplus(dt[:, 0]), 5, name="state")


@pytest.mark.parametrize("d", [256, 37])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_scan_gate(lo, hi, d):
    """B = 0 and D = 1: out is SiLU(z), grad_z its slope."""
    b, t = 3, 100
    z = points(lo, hi, b, t, d)
    zero, skip = torch.zeros(b, t, 1, 1, device="cuda"), torch.ones(d, device="cuda")
    args = scan_of(torch.zeros_like(z), B=zero)
    s, zd = sigmoid(z), z.double()
    with dg.ScanPlan(b, t, d, 1, dtype="fp32") as plan:
        ck = plan.checkpoints()
        within(plan.run(*args, D=skip, z=z, checkpoints=ck), zd * s, 6, name="run")
        g = plan.backward(torch.ones_like(z), *args, ck, D=skip, z=z)
        within(g.z, s + zd * s * (1.0 - s), 8, s + zd.abs() * s * (1.0 - s), "grad_z")
        within(g.u, zd * s, 6, name="grad_u")
        u, dt, A, B, C = (v[:, 0] if v.dim() > 2 else v for v in args)
        cache = torch.zeros(b, d, 1, device="cuda")
        within(plan.step(u, dt, A, B, C, cache, D=skip, z=z[:, 0]), (zd * s)[:, 0], 6, name="step")


@pytest.mark.parametrize("d", [64, 37, 1000, 2050])
@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_norm_gate(act, lo, hi, d):
    """y = 1 without a norm of its own and a residual of 0: r' is the gate's factor; grad_gate its slope."""
    rows = 40
    g = points(lo, hi, rows, d)
    one, zero, w = torch.ones_like(g), torch.zeros_like(g), torch.ones(d, device="cuda")
    s, gd = sigmoid(g), g.double()
    with dg.BlockNormPlan(rows, d, dtype="fp32", gate=act) as plan:
        r, _ = plan.run(one, zero, w, gate=g)
        grad = plan.backward(one, zero, one, zero, w, gate=g)
    if act == "sigmoid":
        within(r, s, 5, name="run")
        within(grad.y, s, 5, name="grad_y")
        if hi <= 0.0:
            within(grad.gate, s * (1.0 - s), 8, name="grad_gate")
    else:
        within(r, gd * s, 6, name="run")
        within(grad.y, gd * s, 6, name="grad_y")
        within(grad.gate, s + gd * s * (1.0 - s), 8, s + gd.abs() * s * (1.0 - s), "grad_gate")


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_far_arguments(dtype):
    """Where the exponential passes the type's range the functions reach their limits, and not-a-number stays so."""
    x = torch.tensor([-1e4, -200.0, -110.0, -104.0, 0.0, 104.0, 200.0, 1e4], device="cuda").repeat(8)[None, None]
    ty = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x = x.to(ty)
    d = x.shape[-1]
    w = torch.tensor([0.0, 1.0], device="cuda").repeat(d, 1)
    with dg.CausalConvPlan(1, 1, d, 2, dtype=dtype) as conv, dg.ScanPlan(1, 1, d, 1, dtype=dtype) as scan, \
            dg.BlockNormPlan(1, d, dtype=dtype, gate="sigmoid") as norm:
        args = (torch.ones_like(x), x, torch.zeros(d, 1, device="cuda"),
                torch.ones(1, 1, 1, 1, device="cuda", dtype=ty), torch.ones(1, 1, 1, 1, device="cuda", dtype=ty))
        one, zero = torch.ones_like(x[0]), torch.zeros_like(x[0])
        for got, want in ((conv.run(x, w), torch.where(x > 0, x, torch.zeros_like(x))),
                          (scan.run(*args), torch.where(x > 0, x, torch.zeros_like(x))),
                          (norm.run(one, zero, w[:, 1].contiguous(), gate=x[0])[0], (x[0] >= 0).to(ty))):
            got, want = got.reshape(-1), want.reshape(-1)
            mid = x.reshape(-1) == 0
            assert torch.equal(got[~mid & (x.reshape(-1).abs() > 120)], want[~mid & (x.reshape(-1).abs() > 120)])
            assert torch.allclose(got[~mid].float(), want[~mid].float(), rtol=1e-6, atol=1e-30)
        bad = torch.full_like(x, float("nan"))
        assert torch.isnan(conv.run(bad, w)).all() and torch.isnan(scan.run(args[0], bad, *args[2:])).all()
        assert torch.isnan(norm.run(one, zero, w[:, 1].contiguous(), gate=bad[0])[0]).all()
