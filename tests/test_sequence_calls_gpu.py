"""How the sequence operators meet the tensors that a program hands them:
layouts that share a buffer."""
import pytest
import torch

import conv2d_backward_implicit_dgrad_gb300 as dg

pytestmark = pytest.mark.gpu


def rand(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def halves(kind, b, t, d, dtype):
    """Two [b, t, d] tensors side by side in one buffer: tokens outside batch rows, or rows a piece of a row apart."""
    if kind == "tokens outside":
        both = torch.zeros(t, b, 2 * d, dtype=dtype, device="cuda").transpose(0, 1)
    else:
        store = torch.zeros(b * (t * 2 * d + 4 * d), dtype=dtype, device="cuda")
        both = store.as_strided((b, t, 2 * d), (t * 2 * d + 4 * d, 2 * d, 1))
    return both[..., :d], both[..., d:], both


@pytest.mark.parametrize("kind", ["tokens outside", "rows apart"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_halves_of_one_buffer(kind, dtype):
    """Input and output, or two outputs, as column halves of one buffer whose batch rows lie inside its tokens."""
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(71)
    b, t, d, n = 3, 40, 24, 16
    w, go = rand(gen, d, 4), rand(gen, b, t, d, dtype=ty)
    data = rand(gen, b, t, d, dtype=ty)
    x, y, both = halves(kind, b, t, d, ty)
    x.copy_(data)
    with dg.CausalConvPlan(b, t, d, 4, dtype=dtype) as plan:
        assert torch.equal(plan.run(x, w, out=y), plan.run(data, w)) and torch.equal(x, data)
        y.zero_()
        got, want = plan.backward(go, x, w, grad_x=y), plan.backward(go, data, w)
        assert torch.equal(got.x, want.x) and torch.equal(got.weight, want.weight) and torch.equal(x, data)
        for shift in (1, d - 1):   # columns that do overlap
            with pytest.raises(dg.DgradError) as e:
                plan.run(x, w, out=both[..., shift:shift + d])
            assert e.value.status == 4
    dt, A, B, C = rand(gen, b, t, d, dtype=ty), -rand(gen, d, n).abs(), rand(gen, b, t, 1, n, dtype=ty), rand(gen, b, t, 1, n, dtype=ty)
    z = rand(gen, b, t, d, dtype=ty)
    with dg.ScanPlan(b, t, d, n, dtype=dtype) as plan:
        ck = plan.checkpoints()
        want = plan.run(data, dt, A, B, C, z=z, checkpoints=ck)
        y.zero_()
        assert torch.equal(plan.run(x, dt, A, B, C, z=z, out=y), want) and torch.equal(x, data)
        want = plan.backward(go, data, dt, A, B, C, ck, z=z)
        gu, gz, both = halves(kind, b, t, d, ty)
        got = plan.backward(go, data, dt, A, B, C, ck, z=z, grad_u=gu, grad_z=gz)
        assert torch.equal(gu, want.u) and torch.equal(gz, want.z) and torch.equal(got.A, want.A)
        with pytest.raises(dg.DgradError) as e:
            plan.backward(go, data, dt, A, B, C, ck, z=z, grad_u=gu, grad_z=both[..., d - 1:2 * d - 1])
        assert e.value.status == 4
