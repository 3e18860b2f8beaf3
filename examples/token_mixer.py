"""A stack of token mixers round short causal convolutions, in 8-bit weights: packed prompts, then tokens one by one.

    python examples/token_mixer.py [--layers 4] [--width 2048] [--prompts 700,64,1500,1] [--steps 64]

A layer takes x and the residual stream h:

    q, s, h = rms_norm_q8(x, residual=h)                  the norm, its 8 bits and the new residual stream
    y = matmul_q8(q, s, W_in)                             query | key | value | gate, and two values a head
    qkv = causal_conv1d(y[qkv], silu)                     4 taps, the last 3 rows carried
    o = gated_delta_rule(qkv, g, beta, normalize=True)    a Dk x Dv state a head, carried
    x = matmul_q8(rms_norm_q8(o * silu(gate)), W_out)

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

    def state(self, slots):
        """Zero states of the convolution and of the delta rule for `slots` requests."""
        device = self.taps.device
        return (torch.zeros(slots, TAPS - 1, self.qkv, dtype=torch.bfloat16, device=device),
                torch.zeros(slots, self.hv, self.dk, self.dv, dtype=torch.float32, device=device))

    def forward(self, x, h, state, seq_offsets, slots):
        """x, h [tokens, width] bfloat16 -> the layer's output and the new residual stream. States move on in place."""
        conv_state, delta_state = state
        hk, hv, dk, dv = self.hk, self.hv, self.dk, self.dv
        q8, scale, h_new = cf.rms_norm_q8(x, self.norm_in, residual=h, out_dtype=self.qtype)
        h = x if h is None else h_new
        y = cf.matmul_q8(q8, scale, *self.w_in)
        qkv, gate, beta, dt = y.split([self.qkv, hv * dv, hv, hv], dim=-1)
        qkv = cf.causal_conv1d(qkv, self.taps, self.taps_bias, activation="silu", seq_offsets=seq_offsets,
                               initial_state=conv_state, final_state=conv_state, slots=slots)
        q, k, v = qkv.split([hk * dk, hk * dk, hv * dv], dim=-1)
        g = self.decay * F.softplus(dt.float() + self.dt_bias)
        o = cf.gated_delta_rule(q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (hv, dv)),
                                g, beta.float().sigmoid(), normalize=True, seq_offsets=seq_offsets,
                                initial_state=delta_state, final_state=delta_state, slots=slots)
        q8, scale, _ = cf.rms_norm_q8(o.flatten(-2) * F.silu(gate), self.norm_out, out_dtype=self.qtype)
        return cf.matmul_q8(q8, scale, *self.w_out), h


class Stack:
    """Layers one after the other, with a state a layer."""

    def __init__(self, layers, slots):
        self.layers, self.states = layers, [layer.state(slots) for layer in layers]

    def run(self, x, seq_offsets, slots):
        h = None
        for layer, state in zip(self.layers, self.states):
            x, h = layer.forward(x, h, state, seq_offsets, slots)
        return x + h


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--heads", default="16,32", help="key heads, value heads")
    ap.add_argument("--prompts", default="700,64,1500,1", help="the prompts' lengths")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--qtype", choices=["int8", "e4m3"], default="int8")
    a = ap.parse_args()
    hk, hv = map(int, a.heads.split(","))
    lens = list(map(int, a.prompts.split(",")))
    n, dev = len(lens), "cuda:0"
    qtype = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[a.qtype]
    stack = Stack([TokenMixer(a.width, hk, hv, 128, 128, qtype, seed=i) for i in range(a.layers)], slots=n)
    slots = torch.arange(n, dtype=torch.int32, device=dev)
    offsets = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().to(dev)
    x = torch.randn(sum(lens), a.width, device=dev).bfloat16()

    def timed(work, times):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(times):
            work()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / times

    stack.run(x, offsets, slots)        # warm
    for state in stack.states:
        state[0].zero_(), state[1].zero_()
    ms = timed(lambda: stack.run(x, offsets, slots), 1)
    print(f"prompts: {sum(lens)} tokens of {n} requests in {ms:.3f} ms, {sum(lens) / ms * 1e3:.0f} tokens/s")

    one = torch.arange(n + 1, dtype=torch.int32, device=dev)
    token = torch.randn(n, a.width, device=dev).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.run(token, one, slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.run(token, one, slots)
    ms = timed(graph.replay, a.steps)
    assert torch.isfinite(out).all()
    print(f"decoding: {a.steps} steps of {n} tokens, {ms * 1e3:.1f} us a step, {n / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
