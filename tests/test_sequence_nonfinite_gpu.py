"""Infinities and not-a-numbers inside a row of the sequence operators: they
reach what the definitions in 64 bits (tests/sequence_batched.py) give them to,
and nothing else.  Finite results keep the bounds of tests/test_sequence_gpu.py.
"""
import pytest
import torch

import conv2d_backward_implicit_dgrad_gb300 as dg
from tests import sequence_batched as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def same_places(got, want, mag, c, name):
    got = got.double()
    fine = torch.isfinite(want)
    wrong = torch.isfinite(got) != fine
    assert not bool(wrong.any()), f"{name}: {int(wrong.sum())} elements finite on one side only"
    off, bound = (got - want).abs()[fine], 2.0 ** -23 * want.abs()[fine] + c * U * mag[fine]
    assert bool((off <= bound).all()), name


def rand(gen, *shape):
    return torch.randn(shape, generator=gen).cuda()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("at", ["first", "middle", "run", "last"])
@pytest.mark.parametrize("d", [24, 37])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_conv(act, d, at, value):
    """One input of one channel, of a row that ends inside the batch's length."""
    gen = torch.Generator().manual_seed(61)
    b, t, k, lens = 3, 61, 4, [61, 29, 0]
    x, gy, w, bias = rand(gen, b, t, d), rand(gen, b, t, d), rand(gen, d, k), rand(gen, d)
    state, gfinal = rand(gen, b, k - 1, d), rand(gen, b, k - 1, d)
    x[1, dict(first=0, middle=13, run=16, last=28)[at], 5] = value
    args = (x, w, bias, lens, state, act, gy, gfinal)
    want, mag = ref.conv(*args), ref.conv(*args, magnitude=True)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    with dg.CausalConvPlan(b, t, d, k, dtype="fp32", activation=act) as plan:
        y = plan.run(x, w, bias=bias, lengths=n, state=state)
        g = plan.backward(gy, x, w, bias=bias, lengths=n, state=state, grad_final_state=gfinal)
    same_places(y, want[0], mag[0], 32, "y")
    same_places(g.x, want[2], mag[2], 64, "grad x")
    same_places(g.weight, want[3], mag[3], 64 + b * t, "grad weight")
    same_places(g.bias, want[4], mag[4], 64 + b * t, "grad bias")
    same_places(g.state, want[5], mag[5], 64, "grad state")


def test_conv_infinite_weight():
    """A tap that meets no token of a row adds nothing to it: 0 tokens times an infinite weight are not a term."""
    gen = torch.Generator().manual_seed(62)
    b, t, d, k, lens = 3, 20, 8, 4, [20, 7, 1]
    x, gy, w = rand(gen, b, t, d), rand(gen, b, t, d), rand(gen, d, k)
    w[3, 0], w[6, 3] = float("inf"), float("-inf")
    args = (x, w, None, lens, torch.ones(b, k - 1, d, device="cuda"), "none", gy, None)
    want, mag = ref.conv(*args), ref.conv(*args, magnitude=True)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    with dg.CausalConvPlan(b, t, d, k, dtype="fp32", activation="none") as plan:
        y = plan.run(x, w, lengths=n, state=args[4])
        g = plan.backward(gy, x, w, lengths=n, state=args[4])
    # (the definition multiplies rows that it pads with zeros; what lies behind a row is 0 by the interface)
    for i, m in enumerate(lens):
        assert torch.count_nonzero(y[i, m:]) == 0 and torch.count_nonzero(g.x[i, m:]) == 0
    # gr[s] = sum over taps k with a token at s + k
    own = torch.zeros(b, t + k - 1, d, dtype=torch.float64, device="cuda")
    for i, m in enumerate(lens):
        for j in range(k):
            own[i, j:j + m] += gy[i, :m].double() * w[:, j].double()
    for i, m in enumerate(lens):
        own[i, k - 1 + m:] = 0.0
    assert torch.equal(torch.isfinite(g.x), torch.isfinite(own[:, k - 1:]))
    assert torch.equal(torch.isfinite(g.state), torch.isfinite(own[:, :k - 1]))


SCAN_INPUTS = ["u", "dt", "B", "C", "z", "go"]


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("what", SCAN_INPUTS)
@pytest.mark.parametrize("t", [26, 400])
def test_scan_stays_in_its_channel_group_and_row(t, what, value):
    """One value of one row: other rows and groups, (for a channel's own inputs) other channels, and the tokens before
    it keep the bits that they have without it, in the outputs; in the gradients, other rows, groups and channels."""
    gen = torch.Generator().manual_seed(63)
    b, d, n, groups, lens = 3, 20, 5, 2, [t, t - 3, 0]
    v = dict(u=rand(gen, b, t, d), dt=rand(gen, b, t, d), B=rand(gen, b, t, groups, n), C=rand(gen, b, t, groups, n),
             z=rand(gen, b, t, d), go=rand(gen, b, t, d))
    A, D, bias, state = -rand(gen, d, n).abs() - 0.05, rand(gen, d), rand(gen, d) - 2.0, rand(gen, b, d, n)
    at = t // 2 + 1
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def both(x):
        with dg.ScanPlan(b, t, d, n, groups=groups, dtype="fp32") as plan:
            ck, final = plan.checkpoints(), torch.empty(b, d, n, device="cuda")
            names = dict(D=D, z=x["z"], dt_bias=bias, lengths=lengths, state=state)
            first = (x["u"], x["dt"], A, x["B"], x["C"])
            out = plan.run(*first, checkpoints=ck, final_state=final, **names)
            return dict(out=out, final=final, **plan.backward(x["go"], *first, ck, **names)._asdict())

    clean = both(v)
    marked = {k: x.clone() for k, x in v.items()}
    if what in ("B", "C"):
        marked[what][0, at, 1, 2] = value
        channel = torch.zeros(d, dtype=torch.bool, device="cuda")
        channel[d // groups:] = True
    else:
        marked[what][0, at, 13] = value
        channel = torch.zeros(d, dtype=torch.bool, device="cuda")
        channel[13] = True
    bad = both(marked)
    assert not torch.isfinite(torch.cat([x[0].flatten() for x in bad.values() if x.dim() == 3])).all()
    for name, x in bad.items():
        y = clean[name]
        if name in ("B", "C"):          # [batch, token, group, state]
            assert torch.equal(x[1:], y[1:]) and torch.equal(x[:, :, 0], y[:, :, 0]), name
        elif name in ("A", "D", "dt_bias"):
            assert torch.equal(x[~channel], y[~channel]), name
        elif name in ("final", "state"):
            assert torch.equal(x[1:], y[1:]) and torch.equal(x[:, ~channel], y[:, ~channel]), name
        else:                           # [batch, token, channel]
            assert torch.equal(x[1:], y[1:]) and torch.equal(x[..., ~channel], y[..., ~channel]), name
            if name == "out":
                assert torch.equal(x[:, :at], y[:, :at]), name


@pytest.mark.parametrize("what", ["u", "dt", "B", "z", "go"])
@pytest.mark.parametrize("t", [26, 400])
def test_scan_not_a_number_reaches_what_depends_on_it(t, what):
    gen = torch.Generator().manual_seed(64)
    b, d, n = 2, 12, 5
    v = dict(u=rand(gen, b, t, d), dt=rand(gen, b, t, d), B=rand(gen, b, t, 1, n), C=rand(gen, b, t, 1, n),
             z=rand(gen, b, t, d), go=rand(gen, b, t, d))
    p = dict(A=-rand(gen, d, n).abs() - 0.05, D=rand(gen, d), dt_bias=rand(gen, d) - 2.0, state=rand(gen, b, d, n))
    v[what][0, t // 2, 0, 0 if what == "B" else ...] = float("nan")
    want, mag = ref.scan(**v, **p), ref.scan(**v, **p, magnitude=True)
    with dg.ScanPlan(b, t, d, n, dtype="fp32") as plan:
        ck, final = plan.checkpoints(), torch.empty(b, d, n, device="cuda")
        names = dict(D=p["D"], z=v["z"], dt_bias=p["dt_bias"], state=p["state"])
        first = (v["u"], v["dt"], p["A"], v["B"], v["C"])
        out = plan.run(*first, checkpoints=ck, final_state=final, **names)
        g = plan.backward(v["go"], *first, ck, **names)
    c = 64 + 4 * t + n
    same_places(out, want[0], mag[0], c, "out")
    same_places(final, want[1], mag[1], c, "final")
    for name in ("u", "dt", "B", "C", "z", "A", "D", "dt_bias", "state"):
        same_places(getattr(g, name), want[2][name], mag[2][name], 2 * c + d + b * t, "grad " + name)


@pytest.mark.parametrize("what", ["u", "B"])
@pytest.mark.parametrize("has_z", [True, False])
@pytest.mark.parametrize("length", [24, 25, 26, 31, 413])
def test_scan_infinite_state_after_the_last_token(length, has_z, what):
    """An infinity that the last token brings in is in no state before a token: grad_A keeps to what it was."""
    gen = torch.Generator().manual_seed(66)
    b, t, d, n, lens = 2, length + 5, 12, 5, [length, length + 5]
    v = dict(u=rand(gen, b, t, d), dt=rand(gen, b, t, d), B=rand(gen, b, t, 1, n), C=rand(gen, b, t, 1, n),
             z=rand(gen, b, t, d) if has_z else None)
    go = rand(gen, b, t, d)
    p = dict(A=-rand(gen, d, n).abs() - 0.05, D=rand(gen, d), dt_bias=rand(gen, d) - 2.0, state=rand(gen, b, d, n))
    v[what][0, length - 1, 0, 0 if what == "B" else ...] = float("inf")
    want = ref.scan(**v, **p, lens=lens, go=go)
    mag = ref.scan(**v, **p, lens=lens, go=go, magnitude=True)
    n_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    with dg.ScanPlan(b, t, d, n, dtype="fp32") as plan:
        ck, final = plan.checkpoints(), torch.empty(b, d, n, device="cuda")
        names = dict(D=p["D"], z=v["z"], dt_bias=p["dt_bias"], state=p["state"], lengths=n_t)
        first = (v["u"], v["dt"], p["A"], v["B"], v["C"])
        out = plan.run(*first, checkpoints=ck, final_state=final, **names)
        g = plan.backward(go, *first, ck, **names)
    assert bool(torch.isfinite(want[2]["A"]).all())
    c = 64 + 4 * t + n
    same_places(out, want[0], mag[0], c, "out")
    same_places(final, want[1], mag[1], c, "final")
    for name in ("u", "dt", "B", "C", "z", "A", "D", "dt_bias", "state"):
        if getattr(g, name) is not None:
            same_places(getattr(g, name), want[2][name], mag[2][name], 2 * c + d + b * t, "grad " + name)


@pytest.mark.parametrize("d", [64, 37, 2051])
def test_norm_keeps_to_its_row(d):
    gen = torch.Generator().manual_seed(65)
    rows = 9
    y, res, gate, gro, gx = (rand(gen, rows, d) for _ in range(5))
    nw, pw, sc = rand(gen, d), rand(gen, d), rand(gen, d)

    def both(y, gate):
        with dg.BlockNormPlan(rows, d, dtype="fp32", gate="silu") as plan:
            r, x = plan.run(y, res, nw, post_weight=pw, gate=gate, scale=sc)
            g = plan.backward(gro, gx, y, res, nw, post_weight=pw, gate=gate, scale=sc)
            return r, x, g.y, g.gate, g.residual

    clean = both(y, gate)
    keep = torch.arange(rows, device="cuda") != 4
    for marked in (0, 1):
        for value in (float("inf"), float("nan")):
            pair = [y.clone(), gate.clone()]
            pair[marked][4, d // 2] = value
            for p, q in zip(both(*pair), clean):
                assert torch.equal(p[keep], q[keep])
