"""The sequence plans' own device memory: its size can be asked for, and a plan
that finds no room has PyTorch give back what it holds unused before it fails."""
import pytest
import torch

import conv2d_backward_implicit_dgrad_gb300 as dg
from conv2d_backward_implicit_dgrad_gb300 import sequence

OOM, INVALID = 5, 1


class FakeCuda:
    def __init__(self):
        self.emptied = 0

    def empty_cache(self):
        self.emptied += 1


class FakeTorch:
    def __init__(self):
        self.cuda = FakeCuda()


def failing(plan, status, times, result):
    """A call that fails `times` times, then returns; counts its calls."""
    calls = []

    def call(c, *args):
        calls.append(args)
        if len(calls) <= times:
            raise dg.DgradError(status, "backward")
        return result

    plan._torch, plan._c, plan._h = FakeTorch(), object(), None
    return call, calls


@pytest.mark.parametrize("kind,cls,n_args,n_results", [("conv", dg.CausalConvPlan, 2 + 1, 4), ("scan", dg.ScanPlan, 7, 9),
                                                       ("norm", dg.BlockNormPlan, 5, 6)])
def test_backward_asks_again_after_pytorch_gave_memory_back(monkeypatch, kind, cls, n_args, n_results):
    class Bind:
        pass

    for status, times, emptied in ((OOM, 0, 0), (OOM, 1, 1), (OOM, 2, 1), (INVALID, 1, 0)):
        plan, bind = object.__new__(cls), Bind()
        call, calls = failing(plan, status, times, tuple(range(n_results)))
        setattr(bind, kind + "_backward", call)
        monkeypatch.setattr(sequence, "_BIND", bind)
        args = tuple(f"tensor {i}" for i in range(n_args))
        if times > emptied or status != OOM:
            with pytest.raises(dg.DgradError) as e:
                plan.backward(*args)
            assert e.value.status == status
        else:
            assert tuple(plan.backward(*args)) == tuple(range(n_results))
        assert plan._torch.cuda.emptied == emptied and len(calls) == 1 + emptied
        assert all(c[:n_args] == args for c in calls)


def grown(call):
    """By how much the device's free memory shrinks during a call, beyond what PyTorch takes for tensors."""
    torch.cuda.synchronize()
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()
    result = call()
    torch.cuda.synchronize()
    return free - torch.cuda.mem_get_info()[0] - (torch.cuda.memory_reserved() - held), result


@pytest.mark.gpu
def test_workspace_is_what_the_plan_says():
    """To within 64 MB (kernels that are loaded meanwhile, the allocation's granularity) of workspaces above 256 MB;
    the parts by the header's formulas."""
    near = 64 << 20
    b, t, d, n = 4, 4096, 4096, 64
    gen = torch.Generator("cuda").manual_seed(81)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    u, dt, B, C, A = rand(b, t, d), rand(b, t, d), rand(b, t, 1, n), rand(b, t, 1, n), -torch.rand(d, n, device="cuda")
    got, plan = grown(lambda: dg.ScanPlan(b, t, d, n))
    chunks = 64 * b * d * 4
    assert plan.workspace_bytes(gradients=False) - chunks * (n + 1) in range(0, 4097)
    assert abs(got - plan.workspace_bytes(gradients=False)) <= near
    ck = plan.checkpoints()
    plan.run(u, dt, A, B, C, checkpoints=ck)
    got, _ = grown(lambda: plan.backward(u, u, dt, A, B, C, ck))
    share = plan.workspace_bytes() - plan.workspace_bytes(gradients=False)
    assert share == chunks * (n + 2) + 32 * 16 * (d // 32) * b * t and share > 4 * near
    assert abs(got - share) <= near
    got, _ = grown(lambda: plan.backward(u, u, dt, A, B, C, ck))
    assert abs(got) <= near
    got, _ = grown(plan.close)
    assert got < -share
    with pytest.raises(ValueError):
        plan.workspace_bytes()
    x, w = rand(2, 600, 512), torch.randn(512, 4, device="cuda")
    with dg.CausalConvPlan(2, 600, 512, 4) as plan:
        parts = max(2 * 3, 768 * torch.cuda.get_device_properties(0).multi_processor_count // 128 + 1 + 2)
        assert plan.workspace_bytes() - plan.workspace_bytes(gradients=False) == 4 * 5 * 512 * parts
        plan.backward(x, x, w)
    with dg.BlockNormPlan(10 ** 6, 512) as plan:
        share = plan.workspace_bytes() - plan.workspace_bytes(gradients=False)
        assert 0 < share <= 12 * 512 * 10 * torch.cuda.get_device_properties(0).multi_processor_count
