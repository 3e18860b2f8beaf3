"""A stack of token mixers round short causal convolutions, in 8-bit weights: packed prompts, then tokens one by one.

    python examples/token_mixer.py [--mixer delta|heads|channels] [--layers 4] [--width 2048] [--prompts 700,64,1500,1]
                                   [--steps 64] [--rotate]

A layer takes x and the residual stream h:

    q, s, h = rms_norm_q8(x, residual=h)                  the norm, its 8 bits and the new residual stream
    y = matmul_q8(q, s, W_in)                             query | key | value | gate, and two values a head
    qkv = causal_conv1d(y[qkv], silu)                     4 taps, the last 3 rows carried
    o = gated_delta_rule(qkv, g, beta, normalize=True)    a Dk x Dv state a head, carried
    x = matmul_q8(rms_norm_q8(o * silu(gate)), W_out)

or, with a selective scan in the delta rule's place,

    y = matmul_q8(q, s, W_in)                             gate | x | b | c, and a step size a head
    xbc = causal_conv1d(y[xbc], silu)
    c, b = rotary(c, positions, k=b)                      their norms for each group, and their rotation by position
    o = selective_scan_heads(x, dt, a, b, c, skip, gate)  a P x N state a head, carried

(--mixer channels: selective_scan, a step size and a state of N for each channel, from a second projection of x, b and c
normed only). With --rotate the delta rule's queries and keys are rotated by position too.

Prompts of several requests are packed into one call. A decoding step has a token of each request, its convolution and
delta states in slots that the requests keep; all layers of a step are one HIP graph. Weights are random.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_forward_amd as cf  # noqa: E402

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TAPS = 4


def quantise(w, dtype):
    """w [N, K] in 8 bits with a scale for each row."""
    scale = w.abs().amax(1) / QMAX[dtype]
    q = w / scale[:, None]
    return (q.round() if dtype == torch.int8 else q).to(dtype), scale


class TokenMixer:
    def __init__(self, width, hk, hv, dk, dv, qtype=torch.int8, seed=0, device="cuda:0"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def rnd(*shape, std=1.0):
            return torch.randn(shape, generator=gen, device=device) * std

        self.hk, self.hv, self.dk, self.dv, self.qtype = hk, hv, dk, dv, qtype
        self.qkv = 2 * hk * dk + hv * dv
        self.norm_in = (1 + rnd(width, std=0.1)).bfloat16()
        self.norm_out = (1 + rnd(hv * dv, std=0.1)).bfloat16()
        self.w_in = quantise(rnd(self.qkv + hv * dv + 2 * hv, width, std=width ** -0.5), qtype)
        self.w_out = quantise(rnd(width, hv * dv, std=(hv * dv) ** -0.5), qtype)
        self.taps, self.taps_bias = rnd(self.qkv, TAPS, std=0.5).bfloat16(), rnd(self.qkv, std=0.1)
        self.decay, self.dt_bias = -(1 + 3 * rnd(hv).abs()), rnd(hv) - 3
        self.frequencies = cf.rotary_frequencies(dk, device=device)[0]

    def state(self, slots):
        """Zero states of the convolution and of the delta rule for `slots` requests."""
        device = self.taps.device
        return (torch.zeros(slots, TAPS - 1, self.qkv, dtype=torch.bfloat16, device=device),
                torch.zeros(slots, self.hv, self.dk, self.dv, dtype=torch.float32, device=device))

    def forward(self, x, h, state, seq_offsets, slots, positions=None):
        """x, h [tokens, width] bfloat16 -> the layer's output and the new residual stream. States move on in place.

        With positions [tokens] queries and keys are rotated by them.
        """
        conv_state, delta_state = state
        hk, hv, dk, dv = self.hk, self.hv, self.dk, self.dv
        q8, scale, h_new = cf.rms_norm_q8(x, self.norm_in, residual=h, out_dtype=self.qtype)
        h = x if h is None else h_new
        y = cf.matmul_q8(q8, scale, *self.w_in)
        qkv, gate, beta, dt = y.split([self.qkv, hv * dv, hv, hv], dim=-1)
        qkv = cf.causal_conv1d(qkv, self.taps, self.taps_bias, activation="silu", seq_offsets=seq_offsets,
                               initial_state=conv_state, final_state=conv_state, slots=slots)
        q, k, v = qkv.split([hk * dk, hk * dk, hv * dv], dim=-1)
        q, k = q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk))
        if positions is not None:
            q, k = cf.rotary(q, positions, self.frequencies, k=k, out=q, k_out=k)
        g = self.decay * F.softplus(dt.float() + self.dt_bias)
        o = cf.gated_delta_rule(q, k, v.unflatten(-1, (hv, dv)),
                                g, beta.float().sigmoid(), normalize=True, seq_offsets=seq_offsets,
                                initial_state=delta_state, final_state=delta_state, slots=slots)
        q8, scale, _ = cf.rms_norm_q8(o.flatten(-2) * F.silu(gate), self.norm_out, out_dtype=self.qtype)
        return cf.matmul_q8(q8, scale, *self.w_out), h


class ScanMixer:
    """A layer with a selective scan: one decay a head, or (channels) one for each channel and state."""

    def __init__(self, width, heads, p, n, groups, qtype=torch.int8, seed=0, channels=False, device="cuda:0"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def rnd(*shape, std=1.0):
            return torch.randn(shape, generator=gen, device=device) * std

        self.heads, self.p, self.n, self.groups, self.qtype, self.channels = heads, p, n, groups, qtype, channels
        self.inner = inner = heads * p
        self.bc = 2 * groups * n
        self.conv = inner if channels else inner + self.bc
        self.norm_in, self.norm_out = ((1 + rnd(k, std=0.1)).bfloat16() for k in (width, inner))
        self.w_in = quantise(rnd(inner + self.conv + (0 if channels else heads), width, std=width ** -0.5), qtype)
        self.w_out = quantise(rnd(width, inner, std=inner ** -0.5), qtype)
        self.taps, self.taps_bias = rnd(self.conv, TAPS, std=0.5).bfloat16(), rnd(self.conv, std=0.1)
        steps = inner if channels else heads
        self.dt_bias, self.skip = rnd(steps) - 4, 1 + rnd(steps, std=0.1)
        self.norm_b, self.norm_c = ((1 + rnd(n, std=0.1)).bfloat16() for _ in range(2))
        self.frequencies = cf.rotary_frequencies(n, device=device)[0]
        if channels:        # step sizes, b and c from a second projection, of the convolution's result
            self.norm_x = (1 + rnd(inner, std=0.1)).bfloat16()
            self.w_x = quantise(rnd(inner + self.bc, inner, std=inner ** -0.5), qtype)
            self.a = -torch.arange(1, n + 1, device=device) * torch.exp(rnd(inner, n, std=0.1))
        else:
            self.a = -(1 + 3 * rnd(heads).abs())

    def state(self, slots):
        """Zero states of the convolution and of the scan for `slots` requests."""
        device = self.taps.device
        shape = (self.inner, self.n) if self.channels else (self.heads, self.p, self.n)
        return (torch.zeros(slots, TAPS - 1, self.conv, dtype=torch.bfloat16, device=device),
                torch.zeros(slots, *shape, dtype=torch.float32, device=device))

    def forward(self, x, h, state, seq_offsets, slots, positions=None):
        """x, h [tokens, width] bfloat16 -> the layer's output and the new residual stream. States move on in place.

        With positions [tokens] b and c are rotated by them (not with a decay for each state: a rotation mixes two states,
        which only together decay as one).
        """
        conv_state, scan_state = state
        inner = self.inner
        seq = dict(seq_offsets=seq_offsets, slots=slots)
        q8, scale, h_new = cf.rms_norm_q8(x, self.norm_in, residual=h, out_dtype=self.qtype)
        h = x if h is None else h_new
        y = cf.matmul_q8(q8, scale, *self.w_in)
        gate, mixed = y[:, :inner], y[:, inner:inner + self.conv]
        mixed = cf.causal_conv1d(mixed, self.taps, self.taps_bias, activation="silu", initial_state=conv_state,
                                 final_state=conv_state, **seq)
        u = mixed[:, :inner]
        if self.channels:
            q8, scale, _ = cf.rms_norm_q8(u, self.norm_x, out_dtype=self.qtype)
            more = cf.matmul_q8(q8, scale, *self.w_x)
            dt, both = more[:, :inner], more[:, inner:]
        else:
            dt, both = y[:, inner + self.conv:], mixed[:, inner:]
        b, c = both.unflatten(-1, (2, self.groups, self.n)).unbind(1)
        if positions is None or self.channels:
            positions = torch.zeros(x.shape[0], dtype=torch.int32, device=x.device)     # norms alone
        c, b = cf.rotary(c, positions, self.frequencies, k=b, q_weight=self.norm_c, k_weight=self.norm_b, out=c, k_out=b)
        kw = dict(skip=self.skip, dt_bias=self.dt_bias, dt_softplus=True, initial_state=scan_state, final_state=scan_state, **seq)
        if self.channels:
            o = cf.selective_scan(u, dt, self.a, b, c, gate=gate, **kw)
        else:
            heads = (self.heads, self.p)
            o = cf.selective_scan_heads(u.unflatten(-1, heads), dt, self.a, b, c, gate=gate.unflatten(-1, heads), **kw).flatten(-2)
        q8, scale, _ = cf.rms_norm_q8(o, self.norm_out, out_dtype=self.qtype)
        return cf.matmul_q8(q8, scale, *self.w_out), h


class Stack:
    """Layers one after the other, with a state a layer."""

    def __init__(self, layers, slots):
        self.layers, self.states = layers, [layer.state(slots) for layer in layers]

    def run(self, x, seq_offsets, slots, positions=None):
        h = None
        for layer, state in zip(self.layers, self.states):
            x, h = layer.forward(x, h, state, seq_offsets, slots, positions)
        return x + h


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--mixer", choices=["delta", "heads", "channels"], default="delta")
    ap.add_argument("--rotate", action="store_true", help="rotate queries and keys (c and b) by position")
    ap.add_argument("--heads", default="16,32", help="key heads (groups), value heads")
    ap.add_argument("--prompts", default="700,64,1500,1", help="the prompts' lengths")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--qtype", choices=["int8", "e4m3"], default="int8")
    a = ap.parse_args()
    hk, hv = map(int, a.heads.split(","))
    lens = list(map(int, a.prompts.split(",")))
    n, dev = len(lens), "cuda:0"
    qtype = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[a.qtype]

    def layer(i):
        if a.mixer == "delta":
            return TokenMixer(a.width, hk, hv, 128, 128, qtype, seed=i)
        if a.mixer == "heads":
            return ScanMixer(a.width, hv, 64, 128, hk, qtype, seed=i)
        return ScanMixer(a.width, hv, 64, 16, 1, qtype, seed=i, channels=True)

    stack = Stack([layer(i) for i in range(a.layers)], slots=n)
    slots = torch.arange(n, dtype=torch.int32, device=dev)
    offsets = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().to(dev)
    x = torch.randn(sum(lens), a.width, device=dev).bfloat16()
    where = torch.cat([torch.arange(m) for m in lens]).to(dev) if a.rotate else None

    def timed(work, times):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(times):
            work()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / times

    stack.run(x, offsets, slots, where)        # warm
    for state in stack.states:
        state[0].zero_(), state[1].zero_()
    ms = timed(lambda: stack.run(x, offsets, slots, where), 1)
    print(f"prompts: {sum(lens)} tokens of {n} requests in {ms:.3f} ms, {sum(lens) / ms * 1e3:.0f} tokens/s")

    one = torch.arange(n + 1, dtype=torch.int32, device=dev)
    token = torch.randn(n, a.width, device=dev).bfloat16()
    where = torch.tensor(lens, device=dev) if a.rotate else None

    def step():
        y = stack.run(token, one, slots, where)
        if where is not None:
            where.add_(1)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    ms = timed(graph.replay, a.steps)
    assert torch.isfinite(out).all()
    print(f"decoding: {a.steps} steps of {n} tokens, {ms * 1e3:.1f} us a step, {n / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
