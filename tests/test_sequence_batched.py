"""The batched 64-bit definitions (tests/sequence_batched.py) against the plain
ones (tests/sequence_reference.py); no GPU."""
import numpy as np
import pytest
import torch

from tests import sequence_batched as batched
from tests import sequence_reference as ref


def same(got, want):
    got = got.numpy()
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= 1e-12 * (1.0 + np.abs(want)))


def to(v):
    return None if v is None else torch.from_numpy(v)


@pytest.mark.parametrize("magnitude", [False, True])
@pytest.mark.parametrize("act,full", [("silu", True), ("none", False)])
def test_conv(act, full, magnitude):
    rng = np.random.default_rng(1)
    b, t, d, k = 4, 9, 5, 3
    lens = [9, 0, 1, 4] if full else None
    x, gy, w = rng.standard_normal((b, t, d)), rng.standard_normal((b, t, d)), rng.standard_normal((d, k))
    bias, st, gf = (rng.standard_normal(s) if full else None for s in ((d,), (b, k - 1, d), (b, k - 1, d)))
    want = ref.conv(x, w, bias, lens, st, act, gy, gf, magnitude=magnitude)
    got = batched.conv(*map(to, (x, w, bias)), lens, to(st), act, to(gy), to(gf), magnitude=magnitude)
    for p, q in zip(got, want):
        same(p, q)


@pytest.mark.parametrize("magnitude", [False, True])
@pytest.mark.parametrize("full", [True, False])
def test_scan(full, magnitude):
    rng = np.random.default_rng(2)
    b, t, d, n, g = 4, 7, 6, 3, 2
    lens = [7, 0, 1, 4] if full else None
    v = dict(u=rng.standard_normal((b, t, d)), dt=rng.standard_normal((b, t, d)), A=-rng.random((d, n)) - 0.1,
             B=rng.standard_normal((b, t, g, n)), C=rng.standard_normal((b, t, g, n)),
             D=rng.standard_normal(d) if full else None, z=rng.standard_normal((b, t, d)) if full else None,
             dt_bias=rng.standard_normal(d) if full else None, state=rng.standard_normal((b, d, n)) if full else None)
    go, gf = rng.standard_normal((b, t, d)), rng.standard_normal((b, d, n)) if full else None
    want = ref.scan(**v, lengths=lens, go=go, gfinal=gf, magnitude=magnitude)
    got = batched.scan(**{k: to(a) for k, a in v.items()}, lens=lens, go=to(go), gfinal=to(gf), magnitude=magnitude)
    same(got[0], want[0])
    same(got[1], want[1])
    for k, a in want[2].items():
        if full or k not in ("z", "D", "dt_bias"):
            same(got[2][k], a)
