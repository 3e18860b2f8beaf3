"""Further token-mixer operators, case by case: inputs, plain forms, definitions in 64 bits, and the bytes and operations
that each one needs.

Three operators that stand after the short causal convolution of a token mixer, beside the gated delta rule:

    rotary  norms of queries and keys for each head, with the rotation by their positions in the same pass
    scan    the selective state space scan with a decay for each channel and state, over packed sequences
    heads   the selective state space scan with one decay a head, over packed sequences

Where ``own`` is false, ``run`` computes an operator with elementary torch operations in 32 bits (angles and long sums
of exponents in 64), rounded once at the end; where it is true, it calls the library.
"""
import math
import random

import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-6
FTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ---- the cases -------------------------------------------------------------------------------------------------------


def listed():
    return [
        # A decoding step of 8 requests somewhere in their answers: one launch's latency.
        dict(name="rotary_decode", op="rotary", seqs=8, tokens=8, ragged=False, hq=32, hk=8, d=128, rotated=128, norm=True,
             interleaved=False, start=1000, scaling="none", dtype="bf16"),
        # A ragged prompt in fp32, half of each head rotated in adjacent pairs, no norm.
        dict(name="rotary_part_f32", op="rotary", seqs=3, tokens=1111, ragged=True, hq=16, hk=16, d=128, rotated=64,
             norm=False, interleaved=True, start=0, scaling="linear", dtype="f32"),
        # Part of a long document, a million tokens in, with frequencies scaled for its length.
        dict(name="rotary_far", op="rotary", seqs=1, tokens=4096, ragged=False, hq=16, hk=2, d=256, rotated=64, norm=True,
             interleaved=False, start=1000003, scaling="parts", dtype="bf16"),
        # A full prefill batch.
        dict(name="rotary_prefill", op="rotary", seqs=7, tokens=16384, ragged=True, hq=32, hk=8, d=128, rotated=128,
             norm=True, interleaved=False, start=0, scaling="none", dtype="bf16"),
        # A decoding step of 64 requests: each one's state moves on by one token.
        dict(name="scan_decode", op="scan", seqs=64, tokens=64, ragged=False, channels=8192, n=16, groups=1, dtype="bf16"),
        # Six packed prompts of uneven lengths, an empty one and a single token among them.
        dict(name="scan_ragged", op="scan", seqs=6, tokens=2047, ragged=True, channels=4096, n=16, groups=1, dtype="bf16"),
        # One long prompt.
        dict(name="scan_prefill", op="scan", seqs=1, tokens=8192, ragged=False, channels=8192, n=16, groups=1, dtype="bf16"),
        # One request's decoding step.
        dict(name="heads_one", op="heads", seqs=1, tokens=1, ragged=False, h=128, p=64, n=128, groups=8, dtype="bf16"),
        # A decoding step of 128 requests: every state is read and written once.
        dict(name="heads_decode", op="heads", seqs=128, tokens=128, ragged=False, h=128, p=64, n=128, groups=8,
             dtype="bf16"),
        # Six packed prompts of uneven lengths, an empty one and a single token among them.
        dict(name="heads_ragged", op="heads", seqs=6, tokens=4095, ragged=True, h=64, p=64, n=128, groups=8, dtype="bf16"),
        # One prompt through a wide layer.
        dict(name="heads_prefill", op="heads", seqs=1, tokens=8192, ragged=False, h=128, p=64, n=128, groups=8,
             dtype="bf16"),
        # One long prompt through a narrow layer: few heads, so the length is what there is to split.
        dict(name="heads_long", op="heads", seqs=1, tokens=16384, ragged=False, h=32, p=64, n=64, groups=1, dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm: an odd multiple of step (the listed cases have the round ones)."""
    return _odd(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step


def _odd(x):
    return max(1, int(x) - 1 + int(x) % 2)


def _sequences(rng, most):
    """(sequences, tokens, ragged): a decoding step, or prompts of equal or uneven lengths."""
    if rng.random() < 0.3:
        seqs = _spread(rng, 1, min(256, max(1, most)))
        return seqs, seqs, False
    seqs = min(_spread(rng, 1, 16), _odd(most))
    tokens = _spread(rng, max(2, seqs), max(2, seqs, most))
    ragged = seqs > 1 and rng.random() < 0.7
    return seqs, tokens if ragged else seqs * _odd(tokens // seqs), ragged


def draw(rng):
    op = rng.choice(["rotary", "scan", "scan", "heads", "heads", "heads"])
    if op == "rotary":
        d = rng.choice([64, 80, 128, 128, 160, 256])
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4])
        dtype = "bf16" if rng.random() < 0.75 else "f32"
        seqs, tokens, ragged = _sequences(rng, 16384 * 40 * 128 * (2 if dtype == "bf16" else 1) // 2 // ((hq + hk) * d))
        return dict(op=op, seqs=seqs, tokens=min(tokens, 16384 * seqs), ragged=ragged, hq=hq, hk=hk, d=d,
                    rotated=rng.choice([d, d, d // 2, d // 4 // 2 * 2]), norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.4, start=_spread(rng, 1, 2000000),
                    scaling=rng.choice(["none", "linear", "parts"]), dtype=dtype)
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    narrow = 1 if dtype == "bf16" else 2
    if op == "scan":
        groups = rng.choice([1, 1, 2])
        channels = _spread(rng, 64, 8192, 8 * groups) + (rng.choice([1, 3]) * groups if rng.random() < 0.15 else 0)
        n = rng.choice([8, 16, 16, 16, 32])
        seqs, tokens, ragged = _sequences(rng, min(16384, 8192 * 8192 * 16 // (channels * n * narrow)))
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, channels=channels, n=n, groups=groups, dtype=dtype)
    groups = rng.choice([1, 1, 2, 4, 8])
    h = groups * rng.choice([1, 2, 5, 8, 16])
    p, n = rng.choice([32, 64, 64, 80, 128]), rng.choice([32, 64, 128, 128, 256])
    seqs, tokens, ragged = _sequences(rng, min(16384, 8192 * 128 * 64 * 128 // (h * p * n * narrow)))
    return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, h=h, p=p, n=n, groups=groups, dtype=dtype)


def lengths(case):
    """The sequences' lengths: equal ones, or uneven ones with an empty sequence and a single token where there is room."""
    n, total = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [total // n] * n
    rng = random.Random(17 * n + total)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if n >= 4:                  # move all of one sequence and all but one token of another to the longest
        order = sorted(range(n), key=lambda i: lens[i])
        a, b, longest = order[0], order[1], order[-1]
        lens[longest] += lens[a] + lens[b] - min(1, lens[b])
        lens[a], lens[b] = 0, min(1, lens[b])
    return lens


# ---- inputs ----------------------------------------------------------------------------------------------------------


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _uniform(gen, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _chunk_plan(lens):
    """Chunks that stay inside a sequence: each one's tokens (-1 past the end), and which chunks come n-th in theirs."""
    c = min(CHUNK, 1 << (max(max(lens), 1) - 1).bit_length())
    rows, order, at = [], [], 0
    for seq, length in enumerate(lens):
        for i in range(-(-length // c)):
            if i == len(order):
                order.append(([], []))
            order[i][0].append(len(rows))
            order[i][1].append(seq)
            rows.append([at + t if t < length else -1 for t in range(i * c, i * c + c)])
        at += length
    rows = torch.tensor(rows, device=DEVICE)
    return rows, [(torch.tensor(a, device=DEVICE), torch.tensor(b, device=DEVICE)) for a, b in order]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=case, lens=lengths(case))
    dt = FTYPE[case["dtype"]]
    op, t = case["op"], case["tokens"]
    s["offsets"] = torch.tensor([0] + s["lens"]).cumsum(0).to(torch.int32).to(DEVICE)
    if op == "rotary":
        hq, hk, d, r = case["hq"], case["hk"], case["d"], case["rotated"]
        # Queries, keys and values as a projection leaves them, in one row; a few strong channels, as trained models have.
        strong = 1.0 + 6.0 * (torch.rand((hq + 2 * hk) * d, generator=gen, device=DEVICE) < 0.02)
        row = (_normal(gen, t, (hq + 2 * hk) * d) * strong).to(dt)
        s["q"] = row[:, :hq * d].view(t, hq, d)
        s["k"] = row[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["q_weight"] = (1.0 + 0.2 * _normal(gen, d)).to(dt) if case["norm"] else None
        s["k_weight"] = (1.0 + 0.2 * _normal(gen, d)).to(dt) if case["norm"] else None
        within = torch.arange(t, device=DEVICE) - torch.repeat_interleave(s["offsets"][:-1].long(),
                                                                          torch.diff(s["offsets"].long()), output_size=t)
        begin = torch.randint(0, 1 + case["start"], (case["seqs"],), generator=gen, device=DEVICE) // 16 + case["start"]
        s["positions"] = within + torch.repeat_interleave(begin, torch.diff(s["offsets"].long()), output_size=t)
        f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEVICE) / r)
        s["scale"] = 1.0
        if case["scaling"] == "linear":
            f = f / 4.0
        elif case["scaling"] == "parts":    # slow frequencies stretched by 32, fast ones kept, a ramp between them
            turns = 4096.0 * f / (2.0 * math.pi)
            keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
            f = f * (keep + (1.0 - keep) / 32.0)
            s["scale"] = 0.1 * math.log(32.0) + 1.0
        s["frequencies"] = f.float()
        return s
    s["plan"] = _chunk_plan(s["lens"])
    groups, n = case["groups"], case["n"]
    wide = case["channels"] if op == "scan" else case["h"] * case["p"]
    steps = case["channels"] if op == "scan" else case["h"]
    # What the convolution before it gives (x, b and c in one row) and what the projection gave (gate and step sizes).
    mixed = torch.nn.functional.silu(_normal(gen, t, wide + 2 * groups * n)).to(dt)
    b = mixed[:, wide:wide + groups * n].view(t, groups, n)
    c = mixed[:, wide + groups * n:].view(t, groups, n)
    other = _normal(gen, t, wide + steps).to(dt)
    s.update(b=b, c=c)
    # Step sizes from a thousandth to a tenth, and decays of a token from e^-0.001 to e^-1.6.
    step = torch.exp(_uniform(gen, math.log(0.001), math.log(0.1), steps))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = other[:, wide:]
    if op == "scan":
        s["x"], s["gate"] = mixed[:, :wide], other[:, :wide]
        s["a"] = -torch.arange(1, n + 1, device=DEVICE) * torch.exp(0.1 * _normal(gen, wide, n))
        s["skip"] = 1.0 + 0.1 * _normal(gen, wide)
        s["state"] = 0.2 * _normal(gen, case["seqs"], wide, n)
    else:
        h, p = case["h"], case["p"]
        s["x"], s["gate"] = mixed[:, :wide].view(t, h, p), other[:, :wide].view(t, h, p)
        s["a"] = -_uniform(gen, 1.0, 16.0, h)
        s["skip"] = 1.0 + 0.1 * _normal(gen, h)
        s["state"] = 0.2 * _normal(gen, case["seqs"], h, p, n)
    s["new_state"] = torch.empty_like(s["state"])
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rotary": _rotary_own, "scan": _scan_own, "heads": _heads_own}[op](s)
    return {"rotary": _rotary_plain, "scan": _scan_plain, "heads": _heads_plain}[op](s)


def _rotary_own(s):
    import convolution_forward_amd as cf
    q, k = cf.rotary(s["q"], s["positions"], s["frequencies"], k=s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                     eps=EPS, interleaved=s["case"]["interleaved"], scale=s["scale"])
    return dict(q=q, k=k)


def _rotary_plain(s):
    r, interleaved = s["case"]["rotated"], s["case"]["interleaved"]
    angle = s["positions"].double()[:, None] * s["frequencies"].double()        # radians; far positions have many turns
    angle = (angle - 2.0 * math.pi * torch.floor(angle / (2.0 * math.pi))).float()
    cos, sin = (s["scale"] * angle.cos())[:, None], (s["scale"] * angle.sin())[:, None]

    def one(x, weight):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * weight.float()
        if interleaved:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
        return torch.cat([turned, y[..., r:]], dim=-1).to(x.dtype)

    return dict(q=one(s["q"], s["q_weight"]), k=one(s["k"], s["k_weight"]))


def _scan_own(s):
    import convolution_forward_amd as cf
    y = cf.selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"],
                          dt_softplus=True, seq_offsets=s["offsets"], initial_state=s["state"], final_state=s["new_state"])
    return dict(y=y, state=s["new_state"])


def _heads_own(s):
    import convolution_forward_amd as cf
    y = cf.selective_scan_heads(s["x"], s["dt"], s["a"], s["b"], s["c"], skip=s["skip"], gate=s["gate"],
                                dt_bias=s["dt_bias"], dt_softplus=True, seq_offsets=s["offsets"], initial_state=s["state"],
                                final_state=s["new_state"])
    return dict(y=y, state=s["new_state"])


def _step_sizes(s):
    v = s["dt"].float() + s["dt_bias"]
    return torch.log1p(torch.exp(-v.abs())) + v.clamp_min(0.0)


def _laid(rows, x):
    """[chunks, tokens of a chunk, ...] in 32 bits; tokens past a sequence's end are zeros (no decay, nothing added)."""
    x = x.float()[rows.clamp_min(0)]
    return x.mul_((rows >= 0).view(rows.shape + (1,) * (x.dim() - 2)))


def _carry(s, decay, added):
    """The state before each chunk, and after each sequence: along a sequence, state * decay + added."""
    start = torch.empty_like(added)
    state = s["state"].clone()
    for chunks, seqs in s["plan"][1]:
        before = state[seqs]
        start[chunks] = before
        state[seqs] = before * decay[chunks] + added[chunks]
    return start, state


def _gated(s, y, rows):
    """Tokens in their order, with the skipped input and the gate, rounded."""
    out = torch.empty(s["x"].shape, device=DEVICE)
    out[rows[rows >= 0]] = y[rows >= 0]
    skip = s["skip"] if s["case"]["op"] == "scan" else s["skip"][:, None]
    g = s["gate"].float()
    out = (out + skip * s["x"].float()) * (g / (1.0 + torch.exp(-g)))
    return out.to(s["x"].dtype)


def _scan_plain(s):
    """All chunks at once, token by token: first for what each adds to the state, then, from the right state, for y."""
    rows = s["plan"][0]
    groups, n = s["case"]["groups"], s["case"]["n"]
    k, c = rows.shape
    x, b, cc = s["x"], _laid(rows, s["b"]), _laid(rows, s["c"])
    d = _step_sizes(s)
    dx = _laid(rows, d * x.float()).view(k, c, groups, -1, 1)
    d = _laid(rows, d).view(k, c, groups, -1, 1)
    a = s["a"].view(groups, -1, n)
    h = torch.zeros((k, groups, a.shape[1], n), device=DEVICE)
    for t in range(c):
        h = h * torch.exp(d[:, t] * a) + dx[:, t] * b[:, t, :, None]
    h, state = _carry(s, torch.exp(d.sum(1) * a).view(k, -1, n), h.view(k, -1, n))
    h = h.view(k, groups, -1, n)
    y = torch.empty((k, c, x.shape[1]), device=DEVICE)
    for t in range(c):
        h = h * torch.exp(d[:, t] * a) + dx[:, t] * b[:, t, :, None]
        y[:, t] = (h * cc[:, t, :, None]).sum(-1).view(k, -1)
    return dict(y=_gated(s, y, rows), state=state)


def _heads_plain(s):
    """By chunks: inside one, a triangle of products; from one to the next, the state is carried."""
    rows, case = s["plan"][0], s["case"]
    per = case["h"] // case["groups"]
    d = _laid(rows, _step_sizes(s))                                                  # [chunks, tokens, heads]
    run_d = (d.double() * s["a"].double()).cumsum(dim=1).movedim(2, 1)               # [chunks, heads, tokens]
    b, c = (_laid(rows, s[i]).movedim(2, 1).contiguous() for i in "bc")              # [chunks, groups, tokens, n]
    dx = (_laid(rows, s["x"]) * d[..., None]).movedim(2, 1).contiguous()             # [chunks, heads, tokens, p]
    lower = torch.ones(rows.shape[1], rows.shape[1], device=DEVICE, dtype=torch.bool).tril()
    within = torch.where(lower, run_d[..., :, None] - run_d[..., None, :], -math.inf).float().exp()
    within *= torch.matmul(c, b.mT.contiguous()).repeat_interleave(per, dim=1)
    to_end = (run_d[..., -1:] - run_d).float().exp()[..., None]
    bh, ch = b.repeat_interleave(per, dim=1), c.repeat_interleave(per, dim=1)
    added = torch.matmul((dx * to_end).mT.contiguous(), bh)                          # [chunks, heads, p, n]
    start, state = _carry(s, run_d[..., -1, None, None].float().exp(), added)
    y = torch.matmul(within, dx) + run_d.float().exp()[..., None] * torch.matmul(ch, start.mT.contiguous())
    return dict(y=_gated(s, y.movedim(1, 2), rows), state=state)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        half = case["rotated"] // 2
        turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device=DEVICE),
                           torch.outer(s["positions"].double(), s["frequencies"].double()))[:, None, :]
        out = {}
        for name in ("q", "k"):
            y = s[name].double().clone()
            weight = s[name + "_weight"]
            if weight is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * weight.double()
            first = torch.arange(half, device=DEVICE)
            at = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
            pair = torch.complex(y[..., at[0]], y[..., at[1]]) * turn
            y[..., at[0]], y[..., at[1]] = pair.real, pair.imag
            out[name] = y
        return out
    # Token by token, all sequences at once, the longest first; a sequence that has ended keeps its state.
    lens = s["lens"]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = s["offsets"].long()[order]
    state = s["state"].double()[order]
    x, b, c = s["x"].double(), s["b"].double(), s["c"].double()
    v = s["dt"].double() + s["dt_bias"].double()
    d = torch.where(v > 0, v + torch.log1p(torch.exp(-v)), torch.log1p(torch.exp(v)))
    a, y = s["a"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device=DEVICE)
    per = (case["channels"] if case["op"] == "scan" else case["h"]) // case["groups"]
    group = torch.arange(per * case["groups"], device=DEVICE) // per
    for t in range(max(lens)):
        live = sum(1 for length in lens if length > t)
        at = start[:live] + t
        bt, ct = b[at][:, group], c[at][:, group]
        if case["op"] == "scan":
            state[:live] = state[:live] * (d[at][..., None] * a).exp() + (d[at] * x[at])[..., None] * bt
            y[at] = (state[:live] * ct).sum(-1)
        else:
            state[:live] *= (d[at] * a).exp()[..., None, None]
            state[:live] += (d[at][..., None] * x[at])[..., None] * bt[:, :, None, :]
            y[at] = torch.matmul(state[:live], ct[..., None])[..., 0]
    g = s["gate"].double()
    y = (y + (s["skip"].double() if case["op"] == "scan" else s["skip"].double()[:, None]) * x) * g * torch.sigmoid(g)
    back = torch.empty(len(lens), dtype=torch.long)
    back[order] = torch.arange(len(lens))
    return dict(y=y, state=state[back.to(DEVICE)])


# ---- what a pass cannot do without -----------------------------------------------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    t = case["tokens"]
    if case["op"] == "rotary":
        n = t * (case["hq"] + case["hk"]) * case["d"]
        turned = t * (case["hq"] + case["hk"]) * case["rotated"]
        return {"bytes": 2 * n * e + 8 * t + 2 * case["rotated"] + (2 * case["d"] * e if case["norm"] else 0),
                "flops": 3 * turned + (4 * n if case["norm"] else 0)}
    groups, n, seqs = case["groups"], case["n"], case["seqs"]
    if case["op"] == "scan":
        c = case["channels"]
        return {"bytes": t * (4 * c + 2 * groups * n) * e + 4 * c * (n + 2) + 8 * seqs * c * n,
                "flops": t * c * (7 * n + 12)}
    h, p = case["h"], case["p"]
    return {"bytes": t * (3 * h * p + h + 2 * groups * n) * e + 12 * h + 8 * seqs * h * p * n,
            "flops": t * h * p * (4 * n + 6)}
