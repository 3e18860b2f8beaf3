"""The selective scans on the GPU against their definitions in 64 bits (scan_ref.py), at the sizes, layouts and values
where they can go wrong."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
import scan_ref as ref
from mixer_ref import seqs
from test_gpu_mixer import BF, DEV, F32, padded, rnd

pytestmark = pytest.mark.gpu
AUTO, DIRECT, TILED = cf.VARIANT_AUTO, cf.VARIANT_DIRECT, cf.VARIANT_TILED


def channel_inputs(tokens, C, G, N, dtype, seed):
    x, dt, gate = (rnd((tokens, C), seed + i, dtype) for i in range(3))
    b, c = (rnd((tokens, G, N), seed + 3 + i, dtype) for i in range(2))
    a = -torch.exp(rnd((C, N), seed + 5))
    return x, dt, a, b, c, rnd(C, seed + 6), gate, rnd(C, seed + 7) - 2.0


def head_inputs(tokens, H, P, G, N, dtype, seed):
    x, gate = (rnd((tokens, H, P), seed + i, dtype) for i in range(2))
    b, c = (rnd((tokens, G, N), seed + 3 + i, dtype) for i in range(2))
    a = -torch.exp(rnd(H, seed + 5))
    return x, rnd((tokens, H), seed + 2, dtype), a, b, c, rnd(H, seed + 6), gate, rnd(H, seed + 7) - 2.0


def gpu(ts):
    return [None if t is None else t.to(DEV) for t in ts]


def run(fn, ins, lens, states, variant=AUTO, softplus=True, **kw):
    """(y, final states) of the call on packed sequences."""
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    st = None if states is None else states.to(DEV)
    shape = (len(lens),) + (tuple(a.shape) if a.dim() == 2 else (a.shape[0], x.shape[-1], b.shape[-1]))
    new = torch.full(shape, float("nan"), device=DEV)
    y = fn(x, dt, a, b, c, skip=skip, gate=gate, dt_bias=bias, dt_softplus=softplus, seq_offsets=seqs(lens, DEV),
           initial_state=st, final_state=new, variant=variant, **kw)
    return y, new


def check(fn, ins, lens, states, variant=AUTO, softplus=True):
    y, new = run(fn, ins, lens, states, variant, softplus)
    define = ref.channels if fn is cf.selective_scan else ref.heads
    y0, by, h0, bh = define(*ins, softplus, lens, states)
    mixer_ref.check(y, y0, by, "y", ins[0].dtype)
    mixer_ref.check(new, h0, bh, "state", F32)


RAGGED = [[1], [5], [3, 0, 1, 9], [64, 63, 65, 1, 0, 2]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", RAGGED, ids=str)
@pytest.mark.parametrize("C,G,N", [(1, 1, 1), (5, 1, 3), (24, 2, 16), (70, 1, 16), (9, 3, 5), (33, 1, 8), (12, 2, 33),
                                   (8, 1, 64), (6, 1, 100), (4, 2, 200), (3, 1, 256)])
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_channels(C, G, N, lens, dtype, variant):
    if variant == TILED and N > 32:
        pytest.skip("tiles take up to 32 states")
    ins = channel_inputs(sum(lens), C, G, N, dtype, C + N)
    check(cf.selective_scan, ins, lens, rnd((len(lens), C, N), 1), variant)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,C,G,N", [([700, 3, 0, 297], 40, 1, 16), ([1000], 20, 2, 8), ([3000], 5, 1, 32),
                                        ([256, 512, 257], 34, 1, 13), ([900, 900], 64, 1, 16)], ids=str)
def test_channels_in_segments(lens, C, G, N, dtype):
    """Sequences past one segment, states updated in place; without offsets where they are equally long."""
    ins, st = channel_inputs(sum(lens), C, G, N, dtype, 21), rnd((len(lens), C, N), 22)
    y0, by, h0, bh = ref.channels(*ins, True, lens, st)
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    kw = dict(skip=skip, dt_bias=bias, dt_softplus=True, variant=TILED)
    pool = st.to(DEV)
    y = cf.selective_scan(x, dt, a, b, c, gate=gate, seq_offsets=seqs(lens, DEV), initial_state=pool, final_state=pool, **kw)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(pool, h0, bh, "state", F32)
    if len(set(lens)) == 1:
        n = len(lens)
        x, dt, b, c, gate = (t.unflatten(0, (n, -1)) for t in (x, dt, b, c, gate))
        pool = st.to(DEV)
        y = cf.selective_scan(x, dt, a, b, c, gate=gate, initial_state=pool, final_state=pool, **kw)
        mixer_ref.check(y.flatten(0, 1), y0, by, "equal, y", dtype)
        mixer_ref.check(pool, h0, bh, "equal, state", F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", RAGGED, ids=str)
@pytest.mark.parametrize("H,P,G,N", [(1, 1, 1, 1), (2, 5, 1, 3), (4, 16, 2, 16), (3, 64, 1, 64), (4, 33, 4, 100), (6, 64, 2, 128),
                                     (2, 80, 1, 30), (2, 128, 2, 200), (1, 24, 1, 256)])
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_heads(H, P, G, N, lens, dtype, variant):
    if variant == TILED and dtype == F32 and N > 128:
        pytest.skip("chunks of fp32 take up to 128 states")
    ins = head_inputs(sum(lens), H, P, G, N, dtype, H + P + N)
    check(cf.selective_scan_heads, ins, lens, rnd((len(lens), H, P, N), 1), variant)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,H,P,G,N", [([700, 3, 0, 297], 2, 32, 1, 64), ([1000], 1, 64, 1, 128), ([5000], 1, 16, 1, 16),
                                          ([256, 512, 257], 3, 40, 3, 128), ([900, 900], 2, 20, 1, 30)], ids=str)
def test_heads_in_segments(lens, H, P, G, N, dtype):
    """Sequences past one segment, states updated in place; without offsets where they are equally long."""
    ins, st = head_inputs(sum(lens), H, P, G, N, dtype, 21), rnd((len(lens), H, P, N), 22)
    y0, by, h0, bh = ref.heads(*ins, True, lens, st)
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    kw = dict(skip=skip, dt_bias=bias, dt_softplus=True, variant=TILED)
    pool = st.to(DEV)
    y = cf.selective_scan_heads(x, dt, a, b, c, gate=gate, seq_offsets=seqs(lens, DEV), initial_state=pool, final_state=pool,
                                **kw)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(pool, h0, bh, "state", F32)
    if len(set(lens)) == 1:
        n = len(lens)
        x, dt, b, c, gate = (t.unflatten(0, (n, -1)) for t in (x, dt, b, c, gate))
        pool = st.to(DEV)
        y = cf.selective_scan_heads(x, dt, a, b, c, gate=gate, initial_state=pool, final_state=pool, **kw)
        mixer_ref.check(y.flatten(0, 1), y0, by, "equal, y", dtype)
        mixer_ref.check(pool, h0, bh, "equal, state", F32)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("drop", ["skip", "gate", "bias", "state", "all"])
def test_optional_inputs(drop, softplus):
    lens = [7, 0, 70]
    for fn, ins, shape in ((cf.selective_scan, channel_inputs(77, 40, 1, 16, BF, 3), (40, 16)),
                           (cf.selective_scan_heads, head_inputs(77, 2, 32, 1, 64, BF, 3), (2, 32, 64))):
        ins = list(ins)
        if not softplus:
            ins[1] = ins[1].abs() * 0.1
            ins[7] = ins[7].abs() * 0.01
        for i, name in ((5, "skip"), (6, "gate"), (7, "bias")):
            if drop in (name, "all"):
                ins[i] = None
        check(fn, ins, lens, None if drop in ("state", "all") else rnd((3,) + shape, 4), softplus=softplus)


def cases():
    return [(cf.selective_scan, channel_inputs(100, 40, 2, 16, BF, 5), (40, 16)),
            (cf.selective_scan_heads, head_inputs(100, 4, 32, 2, 64, BF, 5), (4, 32, 64))]


@pytest.mark.parametrize("which", [0, 1])
def test_views(which):
    """Rows with a pitch and NaN between them give the same bits; what lies between the outputs' rows stays."""
    fn, ins, shape = cases()[which]
    lens, st = [30, 70], rnd((2,) + shape, 6)
    y, new = run(fn, ins, lens, st)
    for extra in (8, 1, 3):
        views = [t if t is None or t.dim() < 2 or i == 2 else padded(t, extra) for i, t in enumerate(ins)]
        out = torch.full(y.shape[:-1] + (y.shape[-1] + extra,), 7.0, dtype=BF, device=DEV)
        y2, new2 = run(fn, views, lens, st, out=out[..., :y.shape[-1]])
        assert torch.equal(y2, y) and torch.equal(new2, new) and (out[..., y.shape[-1]:] == 7).all()


@pytest.mark.parametrize("which", [0, 1])
def test_batches_slots_and_updates_in_place(which):
    fn, ins, shape = cases()[which]
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    kw = dict(skip=skip, dt_bias=bias, dt_softplus=True)
    lens, st = [25] * 4, rnd((4,) + shape, 7).to(DEV)
    y, new = fn(x, dt, a, b, c, gate=gate, seq_offsets=seqs(lens, DEV), initial_state=st, final_state=(z := st.clone()), **kw), z
    four = [t.unflatten(0, (4, 25)) for t in (x, dt, b, c, gate)]
    y4 = fn(four[0], four[1], a, four[2], four[3], gate=four[4], initial_state=st, final_state=(z := st.clone()), **kw)
    assert y4.shape == four[0].shape and torch.equal(y4.flatten(0, 1), y) and torch.equal(z, new)
    # Sequence n in slot [3, -1, 9, 0][n] of five: the third (past the slots) and the second start from zeros, keep nothing.
    slots = torch.tensor([3, -1, 9, 0], dtype=torch.int32, device=DEV)
    pool = torch.full((5,) + shape, 3.0, device=DEV)
    pool[3], pool[0] = st[0], st[3]
    keep = pool.clone()
    ys = fn(x, dt, a, b, c, gate=gate, seq_offsets=seqs(lens, DEV), initial_state=pool, final_state=pool, slots=slots, **kw)
    zero = fn(x, dt, a, b, c, gate=gate, seq_offsets=seqs(lens, DEV), **kw)
    want = torch.cat([y[:25], zero[25:75], y[75:]])
    assert torch.equal(ys, want) and torch.equal(pool[3], new[0]) and torch.equal(pool[0], new[3])
    assert torch.equal(pool[[1, 2, 4]], keep[[1, 2, 4]])


@pytest.mark.parametrize("which", [0, 1])
def test_no_tokens(which):
    """Empty sequences carry their state over; without tokens and states nothing is done."""
    fn, ins, shape = cases()[which]
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    st, new = rnd((2,) + shape, 8).to(DEV), torch.zeros((2,) + shape, device=DEV)
    for variant in (DIRECT, TILED):
        kw = dict(seq_offsets=seqs([0, 0], DEV), variant=variant)
        y = fn(x[:0], dt[:0], a, b[:0], c[:0], initial_state=st, final_state=new, **kw)
        assert y.shape[0] == 0 and torch.equal(new, st)
        fn(x[:0], dt[:0], a, b[:0], c[:0], final_state=new, **kw)
        assert (new == 0).all()
    fn(x[:0], dt[:0], a, b[:0], c[:0])


@pytest.mark.parametrize("which", [0, 1])
def test_rows_behind_the_last_sequence_stay(which):
    fn, ins, shape = cases()[which]
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    for variant in (DIRECT, TILED):
        out, kw = torch.full_like(x, 7.0), dict(seq_offsets=seqs([30, 40], DEV), dt_softplus=True, variant=variant)
        fn(x, dt, a, b, c, out=out, final_state=torch.zeros((2,) + shape, device=DEV), **kw)
        assert (out[70:] == 7).all() and not (out[:70] == 7).all(-1).any()
        assert torch.equal(out[:70], fn(x[:70], dt[:70], a, b[:70], c[:70], **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 37, 63, 64, 99])
@pytest.mark.parametrize("which", ["x", "dt", "b", "c", "state"])
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_channels_not_finite(variant, which, at, value, dtype):
    """What is not finite reaches no earlier token, no other channel (b, c: no other group) and no other sequence."""
    ins = list(channel_inputs(130, 24, 2, 16, dtype, 9))
    lens, st = [100, 30], rnd((2, 24, 16), 10)
    clean, new0 = run(cf.selective_scan, ins, lens, st, variant)
    bad = list(ins)
    i = dict(x=0, dt=1, b=3, c=4).get(which)
    hit = torch.zeros(130, 24, dtype=torch.bool)        # where outputs may differ
    held = torch.zeros(2, 24, dtype=torch.bool)
    if which == "state":
        st = st.clone()
        st[0, 5, 3] = value
        hit[:100, 5] = held[0, 5] = True
    else:
        bad[i] = ins[i].clone()
        if which in ("b", "c"):
            bad[i][at, 1, 2] = value
            hit[at:100 if which == "b" else at + 1, 12:] = True
            held[0, 12:] = which == "b"
        else:
            bad[i][at, 5] = value
            hit[at:100, 5] = held[0, 5] = True
    y, new = run(cf.selective_scan, bad, lens, st, variant)
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit]) and torch.equal(new.cpu()[~held], new0.cpu()[~held])
    if which != "state" and not (which == "dt" and value > 0):      # an infinite step size forgets the state: 0 b x is NaN
        assert not torch.isfinite(y.cpu()[at][hit[at]]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 37, 63, 64, 99])
@pytest.mark.parametrize("which", ["x", "dt", "b", "c", "state"])
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_heads_not_finite(variant, which, at, value, dtype):
    """What is not finite reaches no earlier token, no other row of a head (dt: no other head; b, c: no other group) and
    no other sequence."""
    ins = list(head_inputs(130, 4, 32, 2, 64, dtype, 9))
    lens, st = [100, 30], rnd((2, 4, 32, 64), 10)
    clean, new0 = run(cf.selective_scan_heads, ins, lens, st, variant)
    bad = list(ins)
    i = dict(x=0, dt=1, b=3, c=4).get(which)
    hit = torch.zeros(130, 4, 32, dtype=torch.bool)
    held = torch.zeros(2, 4, 32, dtype=torch.bool)
    if which == "state":
        st = st.clone()
        st[0, 1, 5, 3] = value
        hit[:100, 1, 5] = held[0, 1, 5] = True
    else:
        bad[i] = ins[i].clone()
        if which in ("b", "c"):
            bad[i][at, 1, 2] = value
            hit[at:100 if which == "b" else at + 1, 2:] = True
            held[0, 2:] = which == "b"
        elif which == "dt":
            bad[i][at, 1] = value
            hit[at:100, 1] = held[0, 1] = True
        else:
            bad[i][at, 1, 5] = value
            hit[at:100, 1, 5] = held[0, 1, 5] = True
    y, new = run(cf.selective_scan_heads, bad, lens, st, variant)
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit]) and torch.equal(new.cpu()[~held], new0.cpu()[~held])
    if which != "state" and not (which == "dt" and value > 0):
        assert not torch.isfinite(y.cpu()[at][hit[at]]).any()


def test_strong_decays_and_steps():
    """Steps that forget everything, none at all, and growth: what is forgotten costs the rest no precision."""
    lens = [70, 64]
    for fn, ins, shape in ((cf.selective_scan, channel_inputs(134, 40, 1, 16, F32, 11), (40, 16)),
                           (cf.selective_scan_heads, head_inputs(134, 3, 32, 1, 64, F32, 11), (3, 32, 64))):
        ins = list(ins)
        ins[1] = ins[1].clone()
        ins[1][3] = 200.0
        ins[1][40] = 3000.0
        ins[1][50:60] = -200.0          # steps of zero
        ins[1][66] = 60.0
        for v in (DIRECT, TILED):
            check(fn, ins, lens, rnd((2,) + shape, 12), v)
        ins[1] = ins[1].clamp(-3, 0.5)
        ins[2] = -0.05 * ins[2]         # growth
        for v in (DIRECT, TILED):
            check(fn, ins, lens, rnd((2,) + shape, 12), v)


def test_refusals():
    x, dt, a, b, c, skip, gate, bias = gpu(channel_inputs(20, 24, 2, 16, BF, 13))
    off, st = seqs([20], DEV), torch.zeros(1, 24, 16, device=DEV)
    base = dict(x=x, dt=dt, a=a, b=b, c=c)
    for kw in (dict(x=x.float()), dict(dt=dt[:19]), dict(dt=dt[:, :23]), dict(a=a.bfloat16()), dict(a=a[:23]), dict(a=a.t()),
               dict(b=b[:, 0]), dict(c=c[..., :15]), dict(b=b.float()), dict(skip=skip[:5]), dict(skip=skip.bfloat16()),
               dict(gate=gate[:, :5]), dict(dt_bias=bias[None, :5]), dict(initial_state=st[:, :5]),
               dict(final_state=st.bfloat16()), dict(initial_state=st, final_state=torch.zeros(2, 24, 16, device=DEV)),
               dict(seq_offsets=off.long()), dict(seq_offsets=off[:1]), dict(out=x), dict(out=x.float()),
               dict(slots=off.long()), dict(x=x.t()), dict(b=b[:, :1].expand(20, 5, 16), c=c[:, :1].expand(20, 5, 16)),
               dict(variant=9), dict(final_state=st.transpose(1, 2)),
               dict(workspace=torch.zeros(4, device=DEV))):
        with pytest.raises(ValueError):
            cf.selective_scan(**{**base, **kw})
    x, dt, a, b, c, skip, gate, bias = gpu(head_inputs(20, 4, 32, 2, 64, BF, 13))
    st = torch.zeros(1, 4, 32, 64, device=DEV)
    base = dict(x=x, dt=dt, a=a, b=b, c=c)
    for kw in (dict(x=x.float()), dict(dt=dt[:, :3]), dict(a=a[:3]), dict(a=a.bfloat16()), dict(b=b[:, 0]), dict(c=c[..., :63]),
               dict(b=b.float()), dict(skip=skip[:3]), dict(gate=gate[:, :3]), dict(gate=gate.transpose(1, 2)),
               dict(initial_state=st[..., :63]), dict(out=x), dict(out=x[:, :1].expand_as(x)), dict(seq_offsets=off.long()),
               dict(b=b[:, :1].expand(20, 3, 64), c=c[:, :1].expand(20, 3, 64)), dict(variant=9), dict(x=x[..., 0], dt=dt),
               dict(workspace=torch.zeros(4, device=DEV))):
        with pytest.raises(ValueError):
            cf.selective_scan_heads(**{**base, **kw})


@pytest.mark.parametrize("which", [0, 1])
def test_streams_and_graphs(which):
    """On another stream, and captured with states that move on: every replay equals the same step made eagerly."""
    fn, ins, shape = cases()[which]
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    kw = dict(skip=skip, gate=gate, dt_bias=bias, dt_softplus=True, seq_offsets=seqs([60, 40], DEV))
    st = rnd((2,) + shape, 14).to(DEV)
    eager, live = st.clone(), st.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = fn(x, dt, a, b, c, initial_state=st, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fn(x, dt, a, b, c, initial_state=live, final_state=live, **kw)
    for i in range(4):
        want = fn(x, dt, a, b, c, initial_state=eager, final_state=eager, **kw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(live, eager)
        if i == 0:
            assert torch.equal(first, want)
