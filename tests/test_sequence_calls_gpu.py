"""How the sequence operators meet the tensors that a program hands them:
layouts that share a buffer, version counters."""
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


def test_written_tensors_count_a_version():
    """Every tensor that a call is given to write counts as changed in place, as after torch's own operations."""
    gen = torch.Generator().manual_seed(72)
    b, t, d, n, k = 2, 9, 8, 4, 4
    x, w = rand(gen, b, t, d), rand(gen, d, k)
    buf = {name: torch.empty(b, t, d, device="cuda") for name in ("out", "grad_x", "grad_u", "grad_z")}

    def writes(call, *tensors):
        before = [v._version for v in tensors]
        call()
        assert all(v._version > old for v, old in zip(tensors, before))

    fs, cache, y = torch.empty(b, k - 1, d, device="cuda"), torch.zeros(b, k - 1, d, device="cuda"), torch.empty(b, d, device="cuda")
    with dg.CausalConvPlan(b, t, d, k, dtype="fp32") as plan:
        writes(lambda: plan.run(x, w, out=buf["out"], final_state=fs), buf["out"], fs)
        writes(lambda: plan.backward(x, x, w, grad_x=buf["grad_x"]), buf["grad_x"])
        writes(lambda: plan.step(x[:, 0], w, cache, out=y), cache, y)
    A, B = -rand(gen, d, n).abs(), rand(gen, b, t, 1, n)
    ss = torch.zeros(b, d, n, device="cuda")
    with dg.ScanPlan(b, t, d, n, dtype="fp32") as plan:
        ck = plan.checkpoints()
        writes(lambda: plan.run(x, x, A, B, B, z=x, out=buf["out"], final_state=ss, checkpoints=ck), buf["out"], ss, ck)
        writes(lambda: plan.backward(x, x, x, A, B, B, ck, z=x, grad_u=buf["grad_u"], grad_z=buf["grad_z"]),
               buf["grad_u"], buf["grad_z"])
        writes(lambda: plan.step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], ss, out=y), ss, y)
    r, one = rand(gen, b, d), torch.ones(d, device="cuda")
    a, c = torch.empty(b, d, device="cuda"), torch.empty(b, d, device="cuda")
    e = torch.empty(b, d, device="cuda")
    with dg.BlockNormPlan(b, d, dtype="fp32", gate="silu") as plan:
        writes(lambda: plan.run(r, r, one, gate=r, residual_out=a, out=c), a, c)
        writes(lambda: plan.backward(r, r, r, r, one, gate=r, grad_y=a, grad_gate=c, grad_residual=e), a, c, e)


def test_a_saved_tensor_that_a_call_overwrites_is_noticed():
    gen = torch.Generator().manual_seed(73)
    x, w = rand(gen, 1, 5, 8), rand(gen, 8, 4)
    p = torch.ones(1, 5, 8, device="cuda", requires_grad=True)
    kept = torch.zeros(1, 5, 8, device="cuda")
    loss = (p * kept).sum()               # its backward needs `kept`
    with dg.CausalConvPlan(1, 5, 8, 4, dtype="fp32") as plan:
        plan.run(x, w, out=kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode(), dg.CausalConvPlan(1, 5, 8, 4, dtype="fp32") as plan:
        assert torch.equal(plan.run(x, w, out=torch.empty_like(x)), kept)
