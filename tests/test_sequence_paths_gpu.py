"""The sequence operators at the sizes that take the kernels' other paths, on
the GPU against their batched definitions in 64 bits
(tests/sequence_batched.py): long runs of the convolution, several column
tiles, spans of several chunks, single tokens of many sequences.  Bounds as in
tests/test_sequence_gpu.py.
"""
import pytest
import torch

import conv2d_backward_implicit_dgrad_gb300 as dg
from tests import sequence_batched as ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = {"fp32": 2.0 ** -23, "fp16": 2.0 ** -10, "bf16": 2.0 ** -8}
TINY = {"fp32": 0.0, "fp16": 2.0 ** -24, "bf16": 0.0}
U = 2.0 ** -24


def close(got, want, mag, c, dtype="fp32", name=""):
    """tests/test_sequence_gpu.py's bound, on the GPU."""
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), f"{name}: not finite"
    bound = EPS[dtype] * want.abs() + TINY[dtype] + c * U * mag
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{name}: {float((off / bound.clamp(min=1e-300)).max()):.3g} times the bound"


class Maker:
    def __init__(self, seed, dtype):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.dtype = DT[dtype]

    def f32(self, *shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=self.g, device="cuda") * std + mean

    def act(self, *shape, layout="plain", std=1.0):
        """An activation; 'slice': channels odd elements into a wider row."""
        if layout == "plain":
            return self.f32(*shape, std=std).to(self.dtype)
        return self.f32(*shape[:-1], shape[-1] + 6, std=std).to(self.dtype)[..., 3:3 + shape[-1]]


def lengths_of(ragged, b, t):
    """The rows' lengths: one full, one in the middle of a tile, an empty one, a single token, the others short of full."""
    if not ragged:
        return None, None
    n = ([t, t // 2 + 1, 0, 1] + [t - 3 * i for i in range(b)])[:b]
    return torch.tensor(n, dtype=torch.int32, device="cuda"), n


def poison(t, lens):
    for i, n in enumerate(lens or []):
        t[i, n:] = float("nan")


# With 152 SMs a thread of the convolution walks runs of 64 tokens where that
# still gives 1536 threads an SM, else of 32, 16, 8.  Blocks have 512 channels
# (256 where rows allow no wide access) forwards, 128 (64) backwards.
CONV = [
    # B, L, D, K, dtype, act, ragged, state, layout
    (3, 7001, 1024, 4, "bf16", "silu", True, True, "plain"),     # runs of 16
    (3, 13003, 1024, 3, "fp16", "none", True, True, "plain"),    # runs of 32
    (2, 30011, 1024, 4, "bf16", "silu", False, False, "plain"),  # runs of 64
    (3, 24001, 1028, 2, "fp32", "silu", True, True, "plain"),    # runs of 64, the last block's columns cut off
    (2, 16001, 1025, 4, "fp32", "silu", True, True, "slice"),    # runs of 64, elements one by one
    (3, 4001, 1541, 3, "bf16", "none", True, True, "slice"),     # runs of 16, elements one by one
]


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_runs_and_columns(case):
    b, t, d, k, dtype, act, ragged, has_state, layout = case
    m = Maker(51, dtype)
    x, gy = m.act(b, t, d, layout=layout), m.act(b, t, d, layout=layout)
    w, bias = m.f32(d, k, std=0.5), m.f32(d)
    state, gfinal = (m.act(b, k - 1, d), m.act(b, k - 1, d)) if has_state else (None, None)
    lens_t, lens = lengths_of(ragged, b, t)
    want = ref.conv(x, w, bias, lens, state, act, gy, gfinal)
    mag = ref.conv(x, w, bias, lens, state, act, gy, gfinal, magnitude=True)
    poison(x, lens)
    poison(gy, lens)
    with dg.CausalConvPlan(b, t, d, k, dtype=dtype, activation=act) as plan:
        final = torch.full((b, k - 1, d), float("nan"), dtype=DT[dtype], device="cuda")
        y = plan.run(x, w, bias=bias, lengths=lens_t, state=state, final_state=final)
        g = plan.backward(gy, x, w, bias=bias, lengths=lens_t, state=state, grad_final_state=gfinal)
    close(y, want[0], mag[0], 32, dtype, "y")
    assert torch.equal(final.double(), want[1]), "final state"
    close(g.x, want[2], mag[2], 64, dtype, "grad x")
    close(g.weight, want[3], mag[3], 64 + b * t, "fp32", "grad weight")
    close(g.bias, want[4], mag[4], 64 + b * t, "fp32", "grad bias")
    if has_state:
        close(g.state, want[5], mag[5], 64, dtype, "grad state")


def slots_of(m, s):
    """Slots that s sequences read and others that they write; every fifth is padding, every seventh writes nothing,
    every third writes the slot that it read."""
    p = torch.randperm(2 * s + 3, generator=m.g, device="cuda").to(torch.int32)
    read, write = p[:s].clone(), p[s:2 * s].clone()
    write[::3] = read[::3]
    write[::7] = -1
    read[::5] = -1
    return read, write


@pytest.mark.parametrize("s,d,k,dtype,layout", [(40, 1000, 4, "bf16", "plain"), (33, 1037, 3, "fp16", "slice"),
                                                (21, 2050, 2, "fp32", "plain"), (300, 520, 4, "bf16", "plain")])
def test_conv_step_columns(s, d, k, dtype, layout):
    m = Maker(52, dtype)
    x, w, bias, cache = m.act(s, d, layout=layout), m.f32(d, k, std=0.5), m.f32(d), m.act(2 * s + 3, k - 1, d)
    read, write = slots_of(m, s)
    before = cache.clone()
    with dg.CausalConvPlan(s, 1, d, k, dtype=dtype) as plan:
        y = plan.step(x, w, cache, bias=bias, slots=read, write_slots=write)
        plan.check()
    there = read >= 0
    state = before[read.clamp(min=0).long()]
    args = (x[:, None], w, bias, None, state)
    want, mag = ref.conv(*args), ref.conv(*args, magnitude=True)
    assert torch.count_nonzero(y[~there]) == 0
    close(y[there], want[0][there, 0], mag[0][there, 0], 32, dtype, "y")
    put = there & (write >= 0)
    expect = before.clone()
    expect[write[put].long()] = torch.cat([state[:, 1:], x[:, None]], 1)[put]
    assert torch.equal(cache, expect), "cache"


# A column tile of the scan has 128 channels (64 and fewer above 16 states)
# forwards and, backwards, 256 at up to 4 states, 128 up to 16, 64 up to 32.
# Backwards a block walks a span of several chunks (of the pass before it)
# where those are the finer cut: the two cases of 2048 channels and more,
# with 3 and 2 of them on 152 SMs.
SCAN = [
    # B, L, D, N, groups, dtype, z, ragged, state, layout
    (2, 90, 600, 4, 1, "fp32", True, False, True, "plain"),
    (5, 61, 300, 16, 1, "fp16", True, True, True, "plain"),
    (2, 40, 300, 7, 1, "bf16", True, False, True, "plain"),
    (5, 45, 263, 13, 1, "bf16", True, True, True, "slice"),
    (2, 33, 1030, 2, 2, "fp32", False, False, False, "plain"),
    (2, 50, 200, 30, 1, "fp32", True, False, True, "plain"),
    (2, 777, 515, 13, 1, "fp32", False, False, True, "plain"),
    (5, 400, 650, 16, 2, "fp16", True, True, True, "slice"),
    (8, 512, 2048, 16, 1, "bf16", True, True, True, "plain"),
    (8, 512, 2050, 16, 1, "fp32", True, True, True, "slice"),
    (1, 2048, 4096, 16, 1, "bf16", True, False, True, "plain"),
]


def scan_inputs(m, b, t, d, n, groups, has_z, layout):
    v = dict(u=m.act(b, t, d, layout=layout), dt=m.act(b, t, d, layout=layout, std=0.7),
             B=m.act(b, t, groups * n, layout=layout).unflatten(-1, (groups, n)),
             C=m.act(b, t, groups * n, layout=layout).unflatten(-1, (groups, n)),
             z=m.act(b, t, d, layout=layout) if has_z else None)
    return v, dict(A=-(m.f32(d, n).abs() + 0.05), D=m.f32(d), dt_bias=m.f32(d, mean=-2.0))


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_tiles_and_spans(case):
    b, t, d, n, groups, dtype, has_z, ragged, has_state, layout = case
    m = Maker(53, dtype)
    v, p = scan_inputs(m, b, t, d, n, groups, has_z, layout)
    state, gfinal = (m.f32(b, d, n), m.f32(b, d, n)) if has_state else (None, None)
    go = m.act(b, t, d, layout=layout)
    lens_t, lens = lengths_of(ragged, b, t)
    args = dict(**v, **p, lens=lens, state=state, go=go, gfinal=gfinal)
    want, mag = ref.scan(**args), ref.scan(**args, magnitude=True)
    for x in (*v.values(), go):
        if x is not None:
            poison(x, lens)
    names = dict(D=p["D"], z=v["z"], dt_bias=p["dt_bias"], lengths=lens_t, state=state)
    first = (v["u"], v["dt"], p["A"], v["B"], v["C"])
    with dg.ScanPlan(b, t, d, n, groups=groups, dtype=dtype) as plan:
        final, ck = torch.full((b, d, n), float("nan"), device="cuda"), plan.checkpoints()
        ck.fill_(float("nan"))
        out = plan.run(*first, final_state=final, checkpoints=ck, **names)
        g = plan.backward(go, *first, ck, grad_final_state=gfinal, **names)
    c = 64 + 4 * t + n
    close(out, want[0], mag[0], c, dtype, "out")
    close(final, want[1], mag[1], c, "fp32", "final state")
    per_group = d // groups
    for name, outer, ty in (("u", 0, dtype), ("dt", 0, dtype), ("B", per_group, dtype), ("C", per_group, dtype),
                            ("z", 0, dtype), ("A", b * t, "fp32"), ("D", b * t, "fp32"), ("dt_bias", b * t, "fp32"),
                            ("state", 0, "fp32")):
        if getattr(g, name) is not None:
            close(getattr(g, name), want[2][name], mag[2][name], 2 * c + outer, ty, "grad " + name)


# Where one sequence a block makes more than 8 blocks an SM, a block takes two.
@pytest.mark.parametrize("s,d,n,groups,dtype,layout", [
    (257, 1000, 16, 1, "bf16", "plain"), (131, 1302, 13, 2, "fp16", "slice"), (1001, 66, 40, 1, "fp32", "plain"),
    (255, 1024, 4, 1, "fp32", "plain"), (700, 300, 8, 3, "bf16", "plain")])
def test_scan_step_of_many_sequences(s, d, n, groups, dtype, layout):
    m = Maker(54, dtype)
    v, p = scan_inputs(m, s, 1, d, n, groups, True, layout)
    cache = m.f32(2 * s + 3, d, n)
    read, write = slots_of(m, s)
    before = cache.clone()
    with dg.ScanPlan(s, 1, d, n, groups=groups, dtype=dtype) as plan:
        out = plan.step(v["u"][:, 0], v["dt"][:, 0], p["A"], v["B"][:, 0], v["C"][:, 0], cache, D=p["D"],
                        z=v["z"][:, 0], dt_bias=p["dt_bias"], slots=read, write_slots=write)
        plan.check()
    there = read >= 0
    args = dict(**v, **p, state=before[read.clamp(min=0).long()])
    want, mag = ref.scan(**args), ref.scan(**args, magnitude=True)
    assert torch.count_nonzero(out[~there]) == 0
    close(out[there], want[0][there, 0], mag[0][there, 0], 68 + n, dtype, "out")
    put = there & (write >= 0)
    at = write[put].long()
    close(cache[at], want[1][put], mag[1][put], 68, "fp32", "cache")
    rest = torch.ones(len(cache), dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(cache[rest], before[rest]), "a slot that nobody writes changed"
