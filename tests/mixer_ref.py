"""Token-mixer operators from their definitions in 64 bits on the CPU, each with a bound on how far an fp32 evaluation
may be off (u = 2^-24; gamma(n) = n u / (1 - n u), the classical bound of a sum of n terms in any order).

Nothing here is shared with the library: loops over sequences and tokens, one sum per formula.
"""
import math

import torch

from parity import bf16_spacing

U = 2.0 ** -24
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def gamma(n):
    return n * U / (1 - n * U)


def d(t):
    if t is None:
        return None
    if t.dtype in QMAX:
        return t.cpu().to(torch.float32).double()
    return t.detach().cpu().double()


def half_step(values, dtype):
    """Half the distance between neighbours of `dtype` at each value (0 for float32: its rounding is in the bounds)."""
    if dtype == torch.bfloat16:
        return torch.from_numpy(0.5 * bf16_spacing(values.numpy()))
    if dtype == torch.float8_e4m3fn:        # 3 mantissa bits, subnormal spacing 2^-9
        v = values.abs().clamp_min(2.0 ** -6)
        return 0.5 * torch.exp2(torch.floor(torch.log2(v)) - 3)
    if dtype == torch.int8:
        return torch.full_like(values, 0.5)
    return values.abs() * U


def norm(x, weight, residual, eps):
    """(h, y, relative bound on y): y before quantising. The sum of n squares, its mean, the root and three products."""
    h = x.cpu()
    if residual is not None:
        h = (x.cpu().float() + residual.cpu().float()).to(x.dtype)
    hd = h.double()
    n = x.shape[-1]
    y = hd / (hd.square().mean(-1, keepdim=True) + eps).sqrt() * d(weight)
    return h, y, 0.5 * gamma(n + 2) + 8 * U


def product(x, xs, w, ws, bias):
    """(y, bound) of the scaled product; int8 sums are exact, e4m3 ones are fp32 sums of exact products."""
    a, b = d(x), d(w)
    s = d(xs)[:, None] * d(ws)[None, :]
    y = (a @ b.t()) * s
    size = (a.abs() @ b.abs().t()) * s.abs()
    terms = 2 if x.dtype == torch.int8 else x.shape[1] + 2
    bound = gamma(terms) * size + 3 * U * y.abs()
    if bias is not None:
        y = y + d(bias)
        bound = bound + U * (y.abs() + d(bias).abs())
    return y, bound


def conv(x, w, bias, silu, lens, states, final_rows=True):
    """(y, bound, new states) of the causal convolution over sequences of `lens` rows; states [seqs, taps-1, C] or None."""
    taps, C = w.shape[1], w.shape[0]
    wd, xd = d(w), d(x)
    ys, bs, new, at = [], [], [], 0
    for i, n in enumerate(lens):
        first = torch.zeros(taps - 1, C, dtype=torch.float64) if states is None else d(states[i])
        xx = torch.cat([first, xd[at:at + n]])
        y = torch.zeros(n, C, dtype=torch.float64)
        size = torch.zeros_like(y)
        for j in range(taps):
            y = y + xx[j:j + n] * wd[:, j]
            size = size + (xx[j:j + n] * wd[:, j]).abs()
        if bias is not None:
            y, size = y + d(bias), size + d(bias).abs()
        bound = gamma(taps + 1) * size
        if silu:
            # |silu'| <= 1.1; exp(-y) is off by (|y| + 2) u, the sum and quotient by 3 u
            bound = 1.1 * bound + (y.abs() + 6) * 2 * U * (y * torch.sigmoid(y)).abs()
            y = y * torch.sigmoid(y)
        ys.append(y)
        bs.append(bound)
        new.append(xx[n:])
        at += n
    return torch.cat(ys), torch.cat(bs), torch.stack(new)


def delta(q, k, v, g, beta, scale, normalize, lens, states):
    """(o, bound on o, new states, bound on them).

    The bound follows the rule: with normalised keys and beta <= 1 a step is a contraction of each column of S, so what
    a step adds to a column's error is the rounding of its own terms, at most c u times their sizes, and the decay
    shrinks what came before. c counts a sum over Dk rows, one over a chunk's 64 tokens (a kernel may sum the updates of
    a chunk in any grouping), and the few roundings of the scalars.
    """
    q, k, v, g, beta = d(q), d(k), d(v), d(g), d(beta)
    Hk, Dk = q.shape[1:]
    Hv, Dv = v.shape[1:]
    rep = Hv // Hk
    if normalize:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    c = (Dk + 64 + 16) * U
    o = torch.zeros(v.shape, dtype=torch.float64)
    bo = torch.zeros_like(o)
    new, bnew, at = [], [], 0
    for i, n in enumerate(lens):
        S = torch.zeros(Hv, Dk, Dv, dtype=torch.float64) if states is None else d(states[i]).clone()
        E = torch.zeros(Hv, Dv, dtype=torch.float64)            # error of each column, 2-norm
        for t in range(at, at + n):
            a = torch.exp(g[t])[:, None, None]
            S = a * S
            size = S.square().sum(1).sqrt()
            kn = k[t].square().sum(-1).sqrt()[:, None]
            u = beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
            S = S + k[t][:, :, None] * u[:, None, :]
            terms = size * (1 + beta[t][:, None] * kn * kn) + beta[t][:, None] * v[t].abs() * kn + u.abs() * kn
            E = a[:, 0] * E * (1 + c) + c * terms
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
            qn = scale * q[t].square().sum(-1).sqrt()[:, None]
            bo[t] = qn * (E + c * (size + u.abs() * kn))
        new.append(S)
        bnew.append(E[:, None, :].expand(Hv, Dk, Dv))
        at += n
    return o, bo, torch.stack(new), torch.stack(bnew)


def check(got, want, bound, what, dtype=None):
    """Every value within its bound plus half a step of its type; infinities and NaN in the same places."""
    g = d(got).reshape(want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(g)), f"{what}: not finite at other places"
    lim = bound + half_step(torch.maximum(g.abs(), want.abs())[...].nan_to_num(0, 0, 0), dtype or got.dtype)
    off = ((g - want).abs() - lim)[fine]
    assert off.numel() == 0 or off.max() <= 0, \
        f"{what}: {int((off > 0).sum())} of {off.numel()} values past the bound, worst by {off.max():.3g}"


def seqs(lens, device):
    ends = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return ends.to(device)


def lengths_for(total, n, seed):
    gen = torch.Generator().manual_seed(seed)
    cuts = sorted(torch.randint(0, total + 1, (n - 1,), generator=gen).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


assert math.isclose(gamma(2), 2 * U, rel_tol=1e-6)
