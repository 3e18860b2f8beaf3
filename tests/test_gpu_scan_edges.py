"""The rotary and selective scan operators on the GPU at the edges of what they accept: workspaces, streams, graphs,
segments, far strides, sizes past 2^31 values, and values at fp32's ends."""
import pytest
import torch

import convolution_forward_amd as cf
import mixer_ref
import scan_ref as ref
from mixer_ref import seqs
from test_gpu_mixer import BF, DEV, F32, rnd
from test_gpu_rotary import check as check_rotary
from test_gpu_scan import DIRECT, TILED, channel_inputs, gpu, head_inputs, run

pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("which", ["channels", "heads"])


def case(which, tokens, dtype=BF, seed=50):
    """(operator, inputs, shape of a state, bytes of workspace in `n` sequences) of few channels: cut into segments."""
    if which == "channels":
        def space(n):
            return cf.selective_scan_workspace(tokens, n, 40, 2, 16, dtype=dtype, variant=TILED)
        return cf.selective_scan, channel_inputs(tokens, 40, 2, 16, dtype, seed), (40, 16), space

    def space(n):
        return cf.selective_scan_heads_workspace(tokens, n, 4, 32, 2, 64, dtype=dtype, variant=TILED)
    return cf.selective_scan_heads, head_inputs(tokens, 4, 32, 2, 64, dtype, seed), (4, 32, 64), space


def options(ins):
    x, dt, a, b, c, skip, gate, bias = gpu(ins)
    return (x, dt, a, b, c), dict(skip=skip, gate=gate, dt_bias=bias, dt_softplus=True, variant=TILED)


@BOTH
def test_workspaces(which):
    """A given one, whatever it holds, gives the same bits; one too small, or not of contiguous bytes, is refused."""
    fn, ins, shape, space = case(which, 1000)
    args, kw = options(ins)
    kw |= dict(seq_offsets=seqs([600, 400], DEV), initial_state=rnd((2,) + shape, 51).to(DEV))
    y = fn(*args, final_state=(new := torch.zeros((2,) + shape, device=DEV)), **kw)
    n = space(2)
    assert n > 0
    for fill in (0, 255):       # (255: NaN as floats)
        work = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        got = torch.zeros_like(new)
        assert torch.equal(fn(*args, final_state=got, workspace=work[:n], **kw), y) and torch.equal(got, new)
        assert (work[n:] == fill).all()
    for bad in (work[:n - 1], work[1:n + 1], torch.zeros(2 * n, dtype=torch.uint8, device=DEV)[::2], work[:1].expand(n),
                torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            fn(*args, workspace=bad, **kw)


@BOTH
def test_graphs_that_share_a_workspace(which):
    """Two captured graphs and eager calls, one after the other, in one workspace."""
    fn, ins, shape, space = case(which, 1000)
    args, kw = options(ins)
    kw |= dict(seq_offsets=seqs([600, 400], DEV), workspace=torch.zeros(space(2), dtype=torch.uint8, device=DEV))
    states, graphs, outs = [rnd((2,) + shape, 52 + i).to(DEV) for i in range(3)], [], []
    eager = [s.clone() for s in states]
    fn(*args, **kw)
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fn(*args, initial_state=states[i], final_state=states[i], **kw))
    kw.pop("workspace")
    for _ in range(3):
        want = [fn(*args, initial_state=s, final_state=s, **kw) for s in eager]
        graphs[1].replay()
        y = fn(*args, initial_state=states[2], final_state=states[2], **kw)
        graphs[0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(outs + [y] + states, want + eager))


@BOTH
def test_two_streams_at_once(which):
    """Calls that run side by side have workspaces of their own."""
    fn, ins, shape, _ = case(which, 3000)
    args, kw = options(ins)
    states = [rnd((1,) + shape, 56 + i).to(DEV) for i in range(2)]
    want = [fn(*args, initial_state=s, **dict(kw, seq_offsets=seqs([3000], DEV))) for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    off = seqs([3000], DEV)
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fn(*args, initial_state=states[i], seq_offsets=off, **kw))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[4500, 0, 300, 5000, 1], [4400, 4400]], ids=str)
def test_many_segments(lens, dtype):
    """Heads in more segments than the last kernel puts together by itself; slots, in place, with and without offsets."""
    ins, n = head_inputs(sum(lens), 2, 20, 1, 40, dtype, 58), len(lens)
    st = rnd((n, 2, 20, 40), 59)
    y0, by, h0, bh = ref.heads(*ins, True, lens, st)
    args, kw = options(ins)
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV)
    pool = st.flip(0).to(DEV)
    y = cf.selective_scan_heads(*args, seq_offsets=seqs(lens, DEV), initial_state=pool, final_state=pool, slots=slots, **kw)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(pool.flip(0), h0, bh, "state", F32)
    if len(set(lens)) == 1:
        x, dt, b, c, kw["gate"] = (t.unflatten(0, (n, -1)) for t in (args[0], args[1], args[3], args[4], kw["gate"]))
        pool = st.flip(0).to(DEV)
        y = cf.selective_scan_heads(x, dt, args[2], b, c, initial_state=pool, final_state=pool, slots=slots, **kw)
        mixer_ref.check(y.flatten(0, 1), y0, by, "equal, y", dtype)
        mixer_ref.check(pool.flip(0), h0, bh, "equal, state", F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_whole_sequences_of_many_channels(dtype):
    """Channels (heads) enough for a workgroup a compute unit: long sequences are not cut, and ask for no workspace."""
    lens = [400, 0, 300]
    assert cf.selective_scan_workspace(700, 3, 4100, 1, 5, dtype=dtype, variant=TILED) > 0
    assert cf.selective_scan_workspace(700, 3, 8200, 1, 5, dtype=dtype, variant=TILED) == 0
    ins, st = channel_inputs(700, 8200, 1, 5, dtype, 70), rnd((3, 8200, 5), 71)
    y, new = run(cf.selective_scan, ins, lens, st, TILED)
    y0, by, h0, bh = ref.channels(*ins, True, lens, st)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(new, h0, bh, "state", F32)
    assert cf.selective_scan_heads_workspace(700, 3, 260, 16, 260, 16, dtype=dtype, variant=TILED) == 0
    ins, st = head_inputs(700, 260, 16, 260, 16, dtype, 72), rnd((3, 260, 16, 16), 73)
    y, new = run(cf.selective_scan_heads, ins, lens, st, TILED)
    y0, by, h0, bh = ref.heads(*ins, True, lens, st)
    mixer_ref.check(y, y0, by, "y", dtype)
    mixer_ref.check(new, h0, bh, "state", F32)


@BOTH
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_one_slot_read_by_all(which, variant):
    """Where nothing is written, sequences may begin with one state."""
    fn, ins, shape, _ = case(which, 90)
    args, kw = options(ins)
    kw |= dict(seq_offsets=seqs([50, 0, 40], DEV), variant=variant)
    st = rnd((2,) + shape, 60).to(DEV)
    y = fn(*args, initial_state=st, slots=torch.ones(3, dtype=torch.int32, device=DEV), **kw)
    assert torch.equal(y, fn(*args, initial_state=st[1:].repeat(3, *[1] * len(shape)), **kw))


@BOTH
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_far_rows(which, variant):
    """Rows further apart than the 16-byte forms reach: same bits."""
    fn, ins, shape, _ = case(which, 70)
    args, kw = options(ins)
    kw["variant"] = variant
    off = seqs([3, 67], DEV)
    buf = torch.empty(70, (1 << 22) + 8, dtype=BF, device=DEV)

    def far(t, at):
        view = buf[:, at:at + t[0].numel()].unflatten(-1, t.shape[1:])
        view.copy_(t)
        return view
    y = fn(*args, seq_offsets=off, **kw)
    x, dt, a, b, c = args
    kw["gate"] = far(kw["gate"], 0)
    columns = far(x, 512), far(dt, 1024), a, far(b, 1280), far(c, 1536)
    with pytest.raises(ValueError, match="overlaps"):       # an output among the inputs' columns
        fn(*columns, seq_offsets=off, out=buf[:, 2048:2048 + x[0].numel()].unflatten(-1, x.shape[1:]), **kw)
    out = torch.empty_like(buf)[:, 8:8 + x[0].numel()].unflatten(-1, x.shape[1:])
    got = fn(*columns, seq_offsets=off, out=out, **kw)
    assert torch.equal(got, y) and got.data_ptr() == out.data_ptr()


@BOTH
def test_past_two_to_the_31(which):
    """More values than 32 bits count: the last sequence of a packed call, and its state."""
    T, last = (1 << 17) + 64, 50
    if which == "channels":
        fn, define, ins, shape = cf.selective_scan, ref.channels, list(channel_inputs(last, 16384, 1, 4, BF, 61)), (16384, 4)
    else:
        fn, define, ins, shape = cf.selective_scan_heads, ref.heads, list(head_inputs(last, 128, 128, 1, 16, BF, 61)), (128, 128, 16)
    st = rnd((2,) + shape, 62, F32)
    y0, by, h0, bh = define(*ins, True, [last], st[1:])
    x, dt, a, b, c, skip, gate, bias = gpu(ins)

    def behind(t):
        whole = torch.zeros((T,) + t.shape[1:], dtype=BF, device=DEV)
        whole[-last:] = t
        return whole
    new = st.to(DEV)
    y = fn(behind(x), behind(dt), a, behind(b), behind(c), skip=skip, gate=behind(gate), dt_bias=bias, dt_softplus=True,
           seq_offsets=seqs([T - last, last], DEV), initial_state=new, final_state=new, variant=TILED)
    mixer_ref.check(y[-last:], y0, by, "y", BF)
    mixer_ref.check(new[1:], h0, bh, "state", F32)
    assert (y[:-last] == 0).all()


@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_decay_that_is_no_number(variant):
    """A head's NaN rate stays in its head (a channel's in its channel), from the first token on."""
    for which in ("channels", "heads"):
        fn, ins, shape, _ = case(which, 70)
        lens, st = [70], rnd((1,) + shape, 63)
        clean, new0 = run(fn, ins, lens, st, variant)
        bad = list(ins)
        bad[2] = ins[2].clone()
        bad[2][1] = float("nan")
        y, new = run(fn, bad, lens, st, variant)
        assert torch.isnan(y[:, 1]).all() and torch.isnan(new[0, 1]).all()
        keep = [i for i in range(shape[0]) if i != 1]
        assert torch.equal(y[:, keep], clean[:, keep]) and torch.equal(new[:, keep], new0[:, keep])


@BOTH
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_decay_without_memory(which, variant):
    """A rate of minus infinity forgets the state at every token; one at which nothing of it is left gives the same."""
    fn, ins, shape, _ = case(which, 701)
    ins = list(ins)
    lens, st = [70, 1, 630], rnd((3,) + shape, 69)
    ins[2] = ins[2].clone()
    both = []
    for rate in (-float("inf"), -1e30):
        ins[2][1] = rate
        both.append(run(fn, ins, lens, st, variant))
    assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1])
    assert torch.isfinite(both[0][0]).all() and torch.isfinite(both[0][1]).all()


@BOTH
@pytest.mark.parametrize("variant", [DIRECT, TILED])
def test_values_at_the_end_of_32_bits(which, variant):
    """The largest finite inputs under steps that make them small."""
    fn, ins, shape, _ = case(which, 70, F32)
    ins = list(ins)
    top = torch.finfo(F32).max
    ins[1], ins[7] = ins[1].abs() * 1e-30, None
    for i, at in ((0, (5, 1)), (3, (9, 0)), (4, (11, 0))):
        ins[i] = ins[i].clone()
        ins[i][at] = top if i == 0 else top * 1e-8
    ins[5] = None
    y, new = run(fn, ins, [70], None, variant, softplus=False)
    y0, by, h0, bh = (ref.channels if which == "channels" else ref.heads)(*ins, False, [70], None)
    # Token 11 reads the state that the largest x left, some 3e38 1e-30, with c = 3e30: past fp32's range in any order.
    assert (y0[11, 1].abs().amax() > top) and (y0[:11].abs() < top).all() and (y0[12:].abs() < top).all()
    y[11, 1] = y0[11, 1] = 0
    if which == "heads" and variant == TILED:       # chunks make c . b, here of 3e30 and 3e30, of token 11 and its group
        y[11, :2] = y0[11, :2] = 0
    mixer_ref.check(y, y0, by, "y", F32)
    mixer_ref.check(new, h0, bh, "state", F32)


def test_rotary_past_two_to_the_31():
    T, H, D = (1 << 18) + 8, 64, 128
    q = torch.zeros(T, H, D, dtype=BF, device=DEV)
    f = cf.rotary_frequencies(D, device="cpu")[0]
    w, pos = rnd(D, 64, BF), torch.arange(T)
    ends = torch.tensor([0, 1, T // 2, T - 9, T - 2, T - 1])
    some = rnd((6, H, D), 65, BF)
    q[ends.to(DEV)] = some.to(DEV)
    cf.rotary(q, pos.to(DEV), f.to(DEV), q_weight=w.to(DEV), out=q)
    check_rotary(q[ends.to(DEV)], some, pos[ends], f, w, "ends")
    q[ends.to(DEV)] = 0
    assert (q == 0).all()       # (of either sign: zeros times negative weights)


def test_rotary_captured():
    """Replayed with positions that move on, on another stream, beside eager calls."""
    t, f = 9, cf.rotary_frequencies(64, device=DEV)[0]
    q, k, w = rnd((t, 5, 64), 66, BF).to(DEV), rnd((t, 2, 64), 67, BF).to(DEV), rnd(64, 68, BF).to(DEV)
    pos, graph, side = torch.arange(t, device=DEV), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cf.rotary(q, pos, f, k=k, q_weight=w)
    with torch.cuda.graph(graph):
        a, b = cf.rotary(q, pos, f, k=k, q_weight=w, interleaved=True)
        pos += 1
    for i in range(4):
        now = torch.arange(t, device=DEV, dtype=torch.int32) + i
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
            x, y = cf.rotary(q, now, f, k=k, q_weight=w, interleaved=True)
        torch.cuda.synchronize()
        assert torch.equal(a, x) and torch.equal(b, y)
