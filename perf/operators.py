"""The token-mixer operators, case by case: inputs, plain forms, definitions in 64 bits, and the bytes and operations
that each one needs.

Four operators run one after the other in a token mixer built round a short causal convolution:

    norm     RMS norm with the residual's addition and an output in 8 bits with one scale a token
    product  matrix product of 8-bit operands (int8 or e4m3) with scales for each token and output channel
    conv     causal depthwise convolution over packed sequences, with SiLU and a carried state
    delta    the gated delta rule over packed sequences, with a carried state

Where ``own`` is false, ``run`` computes an operator with elementary torch operations in 32 bits, rounded once at the
end; where it is true, it calls the library.
"""
import math
import random

import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}
QTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
FTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ---- the cases -------------------------------------------------------------------------------------------------------


def listed():
    return [
        # A decoding step of a few requests: one launch's latency.
        dict(name="norm_decode", op="norm", rows=4, width=2048, residual=True, qtype="e4m3", dtype="bf16"),
        # A small prompt without a residual (a model's first norm), rows that fill no power of two.
        dict(name="norm_prompt_int8", op="norm", rows=1000, width=2880, residual=False, qtype="int8", dtype="bf16"),
        # A full prefill batch.
        dict(name="norm_prefill", op="norm", rows=16384, width=4096, residual=True, qtype="e4m3", dtype="bf16"),
        # A decoding step's projection: the weights' bytes are the time.
        dict(name="product_decode", op="product", m=8, n=4096, k=4096, qtype="int8", bias=False, dtype="bf16"),
        # A ragged prompt's projection: no size is a multiple of a tile.
        dict(name="product_ragged_e4m3", op="product", m=1111, n=2200, k=2064, qtype="e4m3", bias=True, dtype="bf16"),
        # A prefill's input projection.
        dict(name="product_prefill", op="product", m=8192, n=8192, k=4096, qtype="int8", bias=False, dtype="bf16"),
        # A decoding step of 64 requests: each sequence's state moves on by one token.
        dict(name="conv_decode", op="conv", seqs=64, tokens=64, ragged=False, channels=8192, taps=4, bias=True,
             dtype="bf16"),
        # Seven packed prompts of uneven lengths.
        dict(name="conv_prefill", op="conv", seqs=7, tokens=8192, ragged=True, channels=8192, taps=4, bias=True,
             dtype="bf16"),
        # One request's decoding step.
        dict(name="delta_one", op="delta", seqs=1, tokens=1, ragged=False, hk=16, hv=32, dk=128, dv=128, dtype="bf16"),
        # A decoding step of 128 requests: every state is read and written once.
        dict(name="delta_decode", op="delta", seqs=128, tokens=128, ragged=False, hk=16, hv=32, dk=128, dv=128,
             dtype="bf16"),
        # Six packed prompts of uneven lengths, an empty one and a single token among them.
        dict(name="delta_ragged", op="delta", seqs=6, tokens=4096, ragged=True, hk=16, hv=32, dk=128, dv=128,
             dtype="bf16"),
        # One long prompt: the longest chain of chunks.
        dict(name="delta_long", op="delta", seqs=1, tokens=16384, ragged=False, hk=16, hv=32, dk=128, dv=128,
             dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm: an odd multiple of step (the listed cases have the round ones)."""
    return _odd(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step


def _odd(x):
    return max(1, int(x) - 1 + int(x) % 2)


def draw(rng):
    op = rng.choice(["norm", "product", "product", "conv", "delta", "delta", "delta"])
    if op == "norm":
        # Widths are those of a model's residual stream: multiples of 8, now and then an odd one.
        width = _spread(rng, 128, 16384, 8) + (rng.choice([1, 3]) if rng.random() < 0.15 else 0)
        dtype = "bf16" if rng.random() < 0.8 else "f32"
        rows = min(_spread(rng, 1, 16384), _odd(16384 * (4096 if dtype == "bf16" else 2048) // width))
        return dict(op=op, rows=rows, width=width, residual=rng.random() < 0.7, qtype=rng.choice(["int8", "e4m3"]),
                    dtype=dtype)
    if op == "product":
        n, k = _spread(rng, 64, 16384, 8), _spread(rng, 128, 8192, 16)
        k += rng.choice([1, 4, 8]) if rng.random() < 0.15 else 0
        m = min(_spread(rng, 1, 16384), _odd(8192 * 8192 * 4096 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, qtype=rng.choice(["int8", "e4m3"]), bias=rng.random() < 0.5,
                    dtype="bf16" if rng.random() < 0.8 else "f32")
    if op == "conv":
        channels = _spread(rng, 64, 16384, 8) + (rng.choice([1, 5]) if rng.random() < 0.15 else 0)
        ragged = rng.random() < 0.6
        seqs = _spread(rng, 1, 64)
        dtype = "bf16" if rng.random() < 0.7 else "f32"
        most = max(seqs, _odd(8192 * (8192 if dtype == "bf16" else 4096) // channels))
        tokens = min(_spread(rng, seqs, 32768), most) if ragged else seqs * min(_spread(rng, 1, 4096), _odd(most // seqs))
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, channels=channels, taps=rng.randint(2, 6),
                    bias=rng.random() < 0.5, dtype=dtype)
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 4])
    dk, dv = rng.choice([64, 96, 128]), rng.choice([64, 80, 128])
    if rng.random() < 0.3:      # decoding
        seqs = min(_spread(rng, 1, 256), _odd(128 * 32 // hv))
        return dict(op=op, seqs=seqs, tokens=seqs, ragged=False, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype)
    seqs = _spread(rng, 1, 16)
    most = (16384 if dtype == "bf16" else 2048) * 16 // max(16, hv)
    tokens = _spread(rng, max(2, seqs), most)
    ragged = seqs > 1 and rng.random() < 0.7
    if not ragged:
        tokens = seqs * _odd(tokens // seqs)
    return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype)


def lengths(case):
    """The sequences' lengths: equal ones, or uneven ones with an empty sequence and a single token where there is room."""
    n, total = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [total // n] * n
    rng = random.Random(31 * n + total)
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


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=case)
    dt = FTYPE[case["dtype"]]
    op = case["op"]
    if op == "norm":
        # A residual stream with a few strong channels, as trained models have them.
        strong = 1.0 + 8.0 * (torch.rand(case["width"], generator=gen, device=DEVICE) < 0.01)
        s["x"] = (_normal(gen, case["rows"], case["width"]) * strong).to(dt)
        s["residual"] = (3.0 * _normal(gen, case["rows"], case["width"]) * strong).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _normal(gen, case["width"])).to(dt)
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]

        def eight(rows):
            v = _normal(gen, rows, k)
            v = v * (QMAX[case["qtype"]] / 4.0)
            v = v.clamp(-QMAX[case["qtype"]], QMAX[case["qtype"]])
            return (v.round() if case["qtype"] == "int8" else v).to(QTYPE[case["qtype"]])

        s["x"], s["w"] = eight(m), eight(n)
        s["x_scale"] = 0.02 + 0.03 * torch.rand(m, generator=gen, device=DEVICE)
        s["w_scale"] = 0.0005 + 0.001 * torch.rand(n, generator=gen, device=DEVICE)
        s["bias"] = _normal(gen, n) if case["bias"] else None
    else:
        lens = lengths(case)
        ends = torch.tensor([0] + lens).cumsum(0)
        s["lens"] = lens
        s["offsets"] = ends.to(torch.int32).to(DEVICE)
        t = case["tokens"]
        if op == "conv":
            c, taps = case["channels"], case["taps"]
            s["x"] = _normal(gen, t, c).to(dt)
            s["w"] = (_normal(gen, c, taps) / math.sqrt(taps)).to(dt)
            s["bias"] = 0.1 * _normal(gen, c) if case["bias"] else None
            s["state"] = _normal(gen, case["seqs"], taps - 1, c).to(dt)
            s["new_state"] = torch.empty_like(s["state"])
        else:
            hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
            # What the convolution before it gives: SiLU of activations, keys and queries still to be normalised,
            # as slices of one buffer whose rows hold 64 more columns that this operator does not read.
            mixed = torch.nn.functional.silu(_normal(gen, t, 2 * hk * dk + hv * dv + 64)).to(dt)
            s["q"] = mixed[:, :hk * dk].view(t, hk, dk)
            s["k"] = mixed[:, hk * dk:2 * hk * dk].view(t, hk, dk)
            s["v"] = mixed[:, 2 * hk * dk:2 * hk * dk + hv * dv].view(t, hv, dv)
            # Decays from a few thousandths to about one a token, by head.
            rate = torch.exp(torch.rand(hv, generator=gen, device=DEVICE) * math.log(16.0))
            s["g"] = -rate * torch.nn.functional.softplus(0.5 * _normal(gen, t, hv) - 4.0)
            s["beta"] = torch.sigmoid(_normal(gen, t, hv))
            s["state"] = 0.2 * _normal(gen, case["seqs"], hv, dk, dv)
            s["new_state"] = torch.empty_like(s["state"])
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _norm_own, "product": _product_own, "conv": _conv_own, "delta": _delta_own}[op](s)
    return {"norm": _norm_plain, "product": _product_plain, "conv": _conv_plain, "delta": _delta_plain}[op](s)


def _norm_own(s):
    import convolution_forward_amd as cf
    q, scale, h = cf.rms_norm_q8(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=QTYPE[s["case"]["qtype"]])
    return _norm_out(s, q, scale, h)


def _norm_out(s, q, scale, h):
    if q.dtype == torch.int8:   # whole numbers stand for multiples of the row's scale
        q = torch.mul(q, scale[:, None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))
    return dict(q=q, scale=scale, **({} if h is None else {"h": h}))


def _norm_plain(s):
    kind = s["case"]["qtype"]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    y = hf * torch.rsqrt((hf * hf).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    top = y.abs().amax(dim=1, keepdim=True)
    y = y * torch.where(top > 0, QMAX[kind] / top, torch.zeros_like(top))
    q = (y.round() if kind == "int8" else y.clamp(-448.0, 448.0)).to(QTYPE[kind])
    return _norm_out(s, q, (top / QMAX[kind])[:, 0], None if s["residual"] is None else h)


def _product_own(s):
    import convolution_forward_amd as cf
    return cf.matmul_q8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out_dtype=FTYPE[s["case"]["dtype"]])


def _product_plain(s):
    y = torch.matmul(s["x"].float(), s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(FTYPE[s["case"]["dtype"]])


def _conv_own(s):
    import convolution_forward_amd as cf
    y = cf.causal_conv1d(s["x"], s["w"], bias=s["bias"], activation="silu", seq_offsets=s["offsets"],
                         initial_state=s["state"], final_state=s["new_state"])
    return dict(y=y, state=s["new_state"])


def _conv_plain(s):
    taps, t = s["case"]["taps"], s["x"].shape[0]
    # Each sequence's carried rows and its tokens one after the other, all sequences in one buffer.
    start = s["offsets"][:-1].long()
    seq = torch.bucketize(torch.arange(t, device=DEVICE), s["offsets"][1:].long(), right=True)
    shift = (taps - 1) * (seq + 1)
    ext = torch.empty((t + (taps - 1) * len(s["lens"]), s["x"].shape[1]), dtype=s["x"].dtype, device=DEVICE)
    first = start + (taps - 1) * torch.arange(len(s["lens"]), device=DEVICE)
    rows = first[:, None] + torch.arange(taps - 1, device=DEVICE)
    at = torch.arange(t, device=DEVICE) + shift
    ext[rows] = s["state"]
    ext[at] = s["x"]
    near = at[:, None] + torch.arange(1 - taps, 1, device=DEVICE)
    y = sum(ext[near[:, j]].float() * s["w"][:, j].float() for j in range(taps))
    if s["bias"] is not None:
        y = y + s["bias"]
    y = y / (1.0 + torch.exp(-y))
    last = first + torch.diff(s["offsets"].long())
    return dict(y=y.to(s["x"].dtype), state=ext[last[:, None] + torch.arange(taps - 1, device=DEVICE)])


def _delta_own(s):
    import convolution_forward_amd as cf
    o = cf.gated_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], normalize=True, seq_offsets=s["offsets"],
                            initial_state=s["state"], final_state=s["new_state"])
    return dict(o=o, state=s["new_state"])


def _unit(x):
    return x * torch.rsqrt((x * x).sum(dim=-1, keepdim=True) + EPS)


def _delta_plain(s):
    """By chunks: inside one, the rule is a triangular system; from one to the next, the state is carried."""
    case, lens = s["case"], s["lens"]
    n, hv, dk, dv = len(lens), case["hv"], case["dk"], case["dv"]
    c = min(CHUNK, 1 << (max(lens) - 1).bit_length())
    chunks = -(-max(lens) // c)
    # Sequences side by side, padded with tokens that change nothing (no decay, beta 0).
    t = case["tokens"]
    seq = torch.bucketize(torch.arange(t, device=DEVICE), s["offsets"][1:].long(), right=True)
    place = seq * (chunks * c) + torch.arange(t, device=DEVICE) - s["offsets"].long()[seq]

    def laid(x):                # [n, heads, chunks, c, ...] in 32 bits
        out = torch.zeros((n * chunks * c,) + x.shape[1:], device=DEVICE)
        out[place] = x.float()
        return out.view((n, chunks, c) + x.shape[1:]).movedim(3, 1).contiguous()

    group = hv // case["hk"]
    q = laid(_unit(s["q"].float())).repeat_interleave(group, dim=1) / math.sqrt(dk)
    k = laid(_unit(s["k"].float())).repeat_interleave(group, dim=1)
    v, g, beta = laid(s["v"]), laid(s["g"]), laid(s["beta"])
    run_g = g.cumsum(dim=-1)
    lower = torch.ones(c, c, device=DEVICE, dtype=torch.bool).tril()
    decay = torch.where(lower, run_g[..., :, None] - run_g[..., None, :], -math.inf).exp()
    a = (beta[..., None] * decay * torch.matmul(k, k.mT.contiguous())).tril(-1)
    within = decay * torch.matmul(q, k.mT.contiguous())
    # The inverse of (1 + a), from blocks of one row to twice as long ones.
    inv = torch.eye(c, device=DEVICE).expand_as(a).contiguous()
    size = 1
    while size < c:
        block = torch.arange(c, device=DEVICE) // size
        low = (block[:, None] % 2 == 1) & (block[None, :] == block[:, None] - 1)
        inv = inv - torch.matmul(inv, torch.matmul(torch.where(low, a, 0.0), inv))
        size *= 2
    up = run_g.exp()[..., None]
    to_end = (run_g[..., -1:] - run_g).exp()[..., None]
    state = s["state"]
    outs = []
    for i in range(chunks):
        u = torch.matmul(inv[:, :, i], beta[:, :, i, :, None] * (v[:, :, i] - up[:, :, i] * torch.matmul(k[:, :, i], state)))
        outs.append(up[:, :, i] * torch.matmul(q[:, :, i], state) + torch.matmul(within[:, :, i], u))
        state = up[:, :, i, -1:] * state + torch.matmul((k[:, :, i] * to_end[:, :, i]).mT.contiguous(), u)
    o = torch.stack(outs, dim=1).movedim(2, 3).reshape(n * chunks * c, hv, dv)
    return dict(o=o[place].to(s["v"].dtype), state=state)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        out = {}
        if s["residual"] is not None:
            out["h"] = x + s["residual"].double()
            x = out["h"].to(s["x"].dtype).double()      # the norm is that of the stored sum
        y = x / ((x ** 2).sum(1, keepdim=True) / case["width"] + EPS).sqrt() * s["weight"].double()
        scale = y.abs().max(1).values / QMAX[case["qtype"]]
        if case["qtype"] == "int8":                     # the multiple of the scale, before its rounding to bf16
            out["q"] = torch.round(y / scale[:, None]) * scale[:, None]
        else:                                           # before the rounding to 8 bits
            out["q"] = y / scale[:, None]
        return dict(out, scale=scale)
    if op == "product":
        x, w = s["x"].to(torch.float32).double(), s["w"].to(torch.float32).double()
        y = (x @ w.t()) * (s["x_scale"].double()[:, None] * s["w_scale"].double()[None, :])
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "conv":
        taps, ys, states, at = case["taps"], [], [], 0
        for i, length in enumerate(s["lens"]):
            xx = torch.cat([s["state"][i], s["x"][at:at + length]]).double()
            y = torch.zeros((length, case["channels"]), device=DEVICE, dtype=torch.float64)
            for j in range(taps):
                y += xx[j:j + length] * s["w"][:, j].double()
            if s["bias"] is not None:
                y += s["bias"].double()
            ys.append(y * torch.sigmoid(y))
            states.append(xx[length:])
            at += length
        return dict(y=torch.cat(ys), state=torch.stack(states))
    # The rule itself, token by token, all sequences and heads at once; a sequence that has ended keeps its state.
    lens, group = s["lens"], case["hv"] // case["hk"]
    lens_d, start = torch.tensor(lens, device=DEVICE), s["offsets"][:-1].long()
    state = s["state"].double()
    o = torch.zeros((case["tokens"], case["hv"], case["dv"]), device=DEVICE, dtype=torch.float64)
    q, k = s["q"].double(), s["k"].double()
    q = (q / (q.square().sum(-1, keepdim=True) + EPS).sqrt() / case["dk"] ** 0.5).repeat_interleave(group, 1)
    k = (k / (k.square().sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(group, 1)
    v, g, beta = s["v"].double(), s["g"].double().exp(), s["beta"].double()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    state, start = state[order], start[order]
    for t in range(max(lens)):
        live = sum(1 for x in lens if x > t)
        at = start[:live] + t
        now = state[:live] * g[at][..., None, None]
        u = beta[at][..., None] * (v[at] - (now * k[at][..., None]).sum(-2))
        now = now + k[at][..., None] * u[..., None, :]
        o[at] = (now * q[at][..., None]).sum(-2)
        state[:live] = now
    back = torch.tensor(order, device=DEVICE).argsort()
    return dict(o=o, state=state[back])


# ---- what a pass cannot do without -----------------------------------------------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        return {"bytes": n * (e * (3 if case["residual"] else 1) + 1) + case["width"] * e + 4 * case["rows"], "flops": 7 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * e + 4 * (m + n + (n if case["bias"] else 0)), "flops": 2 * m * n * k}
    t, n = case["tokens"], case["seqs"]
    if case["op"] == "conv":
        c, taps = case["channels"], case["taps"]
        return {"bytes": 2 * t * c * e + c * taps * e + 2 * n * (taps - 1) * c * e + (4 * c if case["bias"] else 0),
                "flops": t * c * (2 * taps + 4)}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    return {"bytes": t * (2 * hk * dk + 2 * hv * dv) * e + 8 * t * hv + 8 * n * hv * dk * dv, "flops": 6 * t * hv * dk * dv}
