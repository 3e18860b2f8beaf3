"""Head norms with rotation and the selective scans from their definitions in 64 bits on the CPU, each with a bound on how
far an fp32 evaluation may be off (u = 2^-24).

Nothing here is shared with the library: loops over sequences and tokens, one sum per formula.
"""
import torch

from mixer_ref import U, d, gamma


def rotary(x, positions, frequencies, weight, eps, interleaved, scale):
    """(y, bound) for x [tokens, heads, D].

    The norm as in mixer_ref.norm. Cosine and sine of a reduced angle of at most pi/4, itself rounded (0.8 u), come from
    a few products: 4 u each with that; the scale, the products and the sum add 4 u. The angle before its reduction has
    the rounding of three products in 64 bits.
    """
    y = d(x)
    rel = 0.0
    if weight is not None:
        n = x.shape[-1]
        root = (y.square().mean(-1, keepdim=True) + eps).sqrt()
        y = torch.where(y == 0, 0.0, y / root) * d(weight)
        rel = 0.5 * gamma(n + 2) + 8 * U
    bound = rel * y.abs()
    pairs = frequencies.numel()
    angle = positions.cpu().double()[:, None] * d(frequencies)
    cos, sin = scale * angle.cos()[:, None], scale * angle.sin()[:, None]
    first = torch.arange(pairs)
    i, j = (2 * first, 2 * first + 1) if interleaved else (first, first + pairs)
    a, b = y[..., i], y[..., j]
    size = abs(scale) * (a.abs() + b.abs()) * (rel + 8 * U + 4 * 2.0 ** -52 * angle.abs()[:, None])
    y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    bound[..., i], bound[..., j] = size, size
    return y, bound


def _scan(x, dt, a, b, c, skip, gate, bias, softplus, lens, states):
    """x [tokens, C, P], dt [tokens, C], a [C, N] or [C, 1], b and c [tokens, C, N] (of the channel's group): the scan with
    a state [C, P, N], and bounds.

    A step size's relative error rd: the sum v = dt + bias is rounded (u |v|, and softplus' / softplus <= 1), exp(-|v|)
    is off by (|v| + 2) u of it, the rest by 12 u. A decay exp(d a) is off by |d a| (rd + 4 u) + 2 u of it. A step adds
    to a state's error what its own roundings are of `size`, the same sum with all terms positive: rd, the decay's error,
    and 6 u (three roundings token by token; by chunks of 64 a sum of 64 terms and the roundings of its factors, 2 u a
    token and 80 u for an unfinished chunk). An output's sum over N states adds (N + 80) u of its size.
    """
    T, C, P = x.shape
    N = b.shape[-1]
    v = dt if bias is None else dt + bias
    rd = torch.zeros_like(v) + U
    step = v
    if softplus:
        step = v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))
        rd = (2 * v.abs() + 14) * U
    y = torch.zeros(T, C, P, dtype=torch.float64)
    by = torch.zeros_like(y)
    new, bnew, at = [], [], 0
    for i, n in enumerate(lens):
        h = torch.zeros(C, P, N, dtype=torch.float64) if states is None else states[i].clone()
        size, err = h.abs(), torch.zeros_like(h)
        for t in range(at, at + n):
            da = (step[t][:, None] * a)[:, None]                    # [C, 1, N or 1]
            e = torch.exp(da)
            r = rd[t][:, None, None]
            add = (step[t][:, None] * x[t])[..., None] * b[t][:, None]
            h = e * h + add
            size = e * size + add.abs()
            err = e * err + (r + da.abs() * (r + 4 * U) + 6 * U) * size
            y[t] = (h * c[t][:, None]).sum(-1)
            by[t] = ((err + (N + 80) * U * size) * c[t][:, None].abs()).sum(-1)
        new.append(h)
        bnew.append(err + 80 * U * size)
        at += n
    if skip is not None:
        y = y + skip * x
        by = by + 2 * U * ((skip * x).abs() + y.abs())
    if gate is not None:
        s = torch.sigmoid(gate)
        y, by = y * gate * s, by * (gate * s).abs()
        by = by + y.abs() * (2 * gate.abs() + 10) * U
    return y, by, torch.stack(new), torch.stack(bnew)


def channels(x, dt, a, b, c, skip, gate, bias, softplus, lens, states):
    """(y, bound on y, new states, bound on them) of selective_scan; b and c [tokens, groups, N]."""
    per = x.shape[-1] // b.shape[1]
    b, c = (d(t).repeat_interleave(per, 1) for t in (b, c))
    y, by, h, bh = _scan(d(x)[..., None], d(dt), d(a), b, c, None if skip is None else d(skip)[:, None],
                         None if gate is None else d(gate)[..., None], d(bias), softplus, lens,
                         None if states is None else d(states)[:, :, None])
    return y[..., 0], by[..., 0], h[:, :, 0], bh[:, :, 0]


def heads(x, dt, a, b, c, skip, gate, bias, softplus, lens, states):
    """(y, bound on y, new states, bound on them) of selective_scan_heads."""
    per = x.shape[1] // b.shape[1]
    b, c = (d(t).repeat_interleave(per, 1) for t in (b, c))
    return _scan(d(x), d(dt), d(a)[:, None], b, c, None if skip is None else d(skip)[:, None], d(gate), d(bias), softplus,
                 lens, d(states))
