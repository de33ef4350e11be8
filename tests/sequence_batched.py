"""The sequence operators' definitions and gradients in 64 bits for sizes that
tests/sequence_reference.py (one row and token after the other) is too slow
for: the same terms and the same ``magnitude`` rule, all rows at once, as torch
operations on the tensors' device.  Held to that file's values by a CPU test.
"""
import torch


def _d(t):
    return None if t is None else t.detach().double()


def dsilu(x):
    s = torch.sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def dsilu_size(x):
    s = torch.sigmoid(x)
    return s + x.abs() * s * (1.0 - s)


def softplus(x):
    return torch.logaddexp(x, torch.zeros_like(x))


def there(lens, b, t, device):
    """[b, t, 1]: the tokens before each row's end."""
    n = torch.tensor([t] * b if lens is None else [min(max(int(v), 0), t) for v in lens], device=device)
    return (torch.arange(t, device=device)[None] < n[:, None])[..., None], n.tolist()


def conv(x, w, bias=None, lens=None, state=None, act="silu", gy=None, gfinal=None, magnitude=False):
    """y, final state and, with gy, the gradients (gx, gw, gbias, gstate)."""
    f = torch.abs if magnitude else (lambda v: v)
    x, w, bias, state, gy, gfinal = map(_d, (x, w, bias, state, gy, gfinal))
    b, t, d = x.shape
    k = w.shape[1]
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    on, n = there(lens, b, t, x.device)
    rows = torch.cat([torch.zeros(b, k - 1, d, dtype=torch.float64, device=x.device) if state is None else state,
                      torch.where(on, x, zero)], 1)
    final = torch.stack([rows[i, m:m + k - 1] for i, m in enumerate(n)])
    pre = sum(rows[:, j:j + t] * w[:, j] for j in range(k)) + (0.0 if bias is None else bias)
    size = sum((rows[:, j:j + t] * w[:, j]).abs() for j in range(k)) + (0.0 if bias is None else bias.abs())
    if act == "silu":
        y = size * (1.0 + pre.abs()) if magnitude else pre * torch.sigmoid(pre)
    else:
        y = size if magnitude else pre
    y = torch.where(on, y, zero)
    if gy is None:
        return y, final
    q = f(gy)
    if act == "silu":
        q = q * ((dsilu(pre).abs() + size + 1.0) if magnitude else dsilu(pre))
    gr = torch.zeros_like(rows)
    gw = torch.zeros_like(w)
    for j in range(k):
        gr[:, j:j + t] += torch.where(on, q * f(w[:, j]), zero)
        gw[:, j] = torch.where(on, q * f(rows[:, j:j + t]), zero).sum((0, 1))
    gb = torch.where(on, q, zero).sum((0, 1))
    if gfinal is not None:
        for i, m in enumerate(n):
            gr[i, m:m + k - 1] += f(gfinal[i])
    gx = torch.where(on, gr[:, k - 1:], zero)
    return y, final, gx, gw, gb, gr[:, :k - 1]


def scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, lens=None, state=None, go=None, gfinal=None, magnitude=False):
    """out, final state and, with go, a dict of the gradients."""
    f = torch.abs if magnitude else (lambda v: v)
    u, dt, A, B, C, D, z, dt_bias, state, go, gfinal = map(_d, (u, dt, A, B, C, D, z, dt_bias, state, go, gfinal))
    b, t, d = u.shape
    g, n = B.shape[2:]
    dev = dict(dtype=torch.float64, device=u.device)
    zero = torch.zeros((), **dev)
    on, _ = there(lens, b, t, u.device)
    skip = torch.zeros(d, **dev) if D is None else f(D)
    off = 0.0 if dt_bias is None else dt_bias
    us, x = torch.where(on, f(u), zero), torch.where(on, dt + off, zero)
    delta, slope = torch.where(on, softplus(x), zero), torch.sigmoid(x)
    Bs, Cs = torch.where(on[..., None], f(B), zero), torch.where(on[..., None], f(C), zero)

    def wide(v):   # [b, groups, states] to [b, channels, states]
        return v.repeat_interleave(d // g, 1)

    def decay(s):
        return torch.exp(delta[:, s, :, None] * A)

    gate = None if z is None else torch.where(on, f(z * torch.sigmoid(z)), zero)
    h = torch.zeros(b, d, n, **dev) if state is None else f(state)
    hs, ys, out = [h], [], torch.zeros(b, t, d, **dev)
    for s in range(t):
        h = decay(s) * h + (delta[:, s] * us[:, s])[..., None] * wide(Bs[:, s])
        y = (h * wide(Cs[:, s])).sum(-1) + skip * us[:, s]
        out[:, s] = torch.where(on[:, s], y if z is None else y * gate[:, s], zero)
        if go is not None:
            hs.append(h)
            ys.append(y)
    if go is None:
        return out, h
    gs = torch.where(on, f(go), zero)
    gr = {k: torch.zeros(v, **dev) for k, v in dict(u=u.shape, dt=u.shape, z=u.shape, A=A.shape, B=B.shape, C=B.shape,
                                                    D=(d,), dt_bias=(d,)).items()}
    back = torch.zeros(b, d, n, **dev) if gfinal is None else f(gfinal)
    for s in reversed(range(t)):
        a, Bt, Ct = decay(s), wide(Bs[:, s]), wide(Cs[:, s])
        dy = gs[:, s] if z is None else gs[:, s] * gate[:, s]
        if z is not None:
            zs = torch.where(on[:, s], z[:, s], zero)
            gr["z"][:, s] = torch.where(on[:, s], gs[:, s] * (dsilu_size(zs) if magnitude else dsilu(zs)) * ys[s], zero)
        gt = dy[..., None] * Ct + back
        per = (gt * Bt).sum(-1)
        through = gt * a * hs[s]
        gr["u"][:, s] = per * delta[:, s] + skip * dy
        gr["dt"][:, s] = torch.where(on[:, s], (per * us[:, s] + (through * f(A)).sum(-1)) * slope[:, s], zero)
        gr["A"] += torch.where(on[:, s, :, None], through * delta[:, s, :, None], zero).sum(0)
        gr["D"] += torch.where(on[:, s], dy * us[:, s], zero).sum(0)
        gr["B"][:, s] = torch.where(on[:, s, :, None], (gt * (delta[:, s] * us[:, s])[..., None]).unflatten(1, (g, d // g)).sum(2), zero)
        gr["C"][:, s] = torch.where(on[:, s, :, None], (dy[..., None] * hs[s + 1]).unflatten(1, (g, d // g)).sum(2), zero)
        back = gt * a
    gr["dt_bias"] = gr["dt"].sum((0, 1))
    gr["state"] = back
    return out, h, gr
