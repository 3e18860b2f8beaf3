"""The selective scans and the rotation together with the other token-mixer operators, as examples/token_mixer.py runs them."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from test_gpu_token_mixer import DEV, offsets, token_mixer

pytestmark = pytest.mark.gpu


def layer(kind, qtype):
    if kind == "delta":
        return token_mixer.TokenMixer(256, 2, 4, 128, 64, qtype, seed=3)
    if kind == "heads":
        return token_mixer.ScanMixer(256, 4, 64, 64, 2, qtype, seed=3)
    return token_mixer.ScanMixer(256, 4, 64, 16, 1, qtype, seed=3, channels=True)


@pytest.mark.parametrize("qtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("kind", ["delta", "heads", "channels"])
def test_prompt_then_single_tokens(kind, qtype):
    """A prompt in one call (chunks, tiles) equals the same prompt cut, its last tokens one by one, with their positions.

    Sums in another order turn a bf16 rounding now and then, and with it a row's scale by 2^-8 and 8-bit values by a step
    each: 1/127 of the row's largest (1/16 of the value itself in e4m3), some 3 times the row's RMS. Such steps at random in
    all K places leave about 2 % of the outputs' RMS; 5 deviations of it are 0.1, and the two projections after another
    that the channel form has 0.15. States hold such values (2^-6 with room; a second projection's, 2^-4).
    """
    lens, last = [150, 70, 1, 0, 33], [6, 6, 1, 0, 6]
    n = len(lens)
    mixer = layer(kind, qtype)
    x = torch.randn(sum(lens), 256, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    where = torch.cat([torch.arange(m) + 1000 * i for i, m in enumerate(lens)]).to(DEV)
    slots = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32, device=DEV)
    whole, cut = mixer.state(n), mixer.state(n)
    want, _ = mixer.forward(x, None, whole, offsets(lens), slots, where)
    rows = list(torch.arange(sum(lens), device=DEV).split(lens))
    got = torch.zeros_like(want)

    def step(index, counts):
        got[index], _ = mixer.forward(x[index], None, cut, offsets(counts), slots, where[index])

    head = [a - b for a, b in zip(lens, last)]
    step(torch.cat([r[:m] for r, m in zip(rows, head)]), head)
    for t in range(max(last)):
        counts = [int(t < b) for b in last]
        step(torch.cat([r[m + t:m + t + c] for r, m, c in zip(rows, head, counts)]), counts)
    rms = want.double().square().mean().sqrt()
    twice = kind == "channels"
    assert torch.isfinite(want).all() and rms > 0
    assert ((got.double() - want.double()).abs().max() / rms).item() <= (0.15 if twice else 0.1)
    for a, b, part in zip(cut, whole, (2 ** -6, 2 ** -4 if twice else 2 ** -6)):
        assert (a.float() - b.float()).abs().max().item() <= part * b.float().abs().max().item()


def test_positions_count():
    """With one decay a head the outputs depend on where tokens are relative to each other only, since c . b does, up to
    roundings of b and c in bf16 (with a decay for each state they would not: its pairs do not decay as one)."""
    mixer = layer("heads", torch.int8)
    x = torch.randn(90, 256, generator=torch.Generator().manual_seed(6)).bfloat16().to(DEV)
    at = torch.arange(90, device=DEV)

    def run(where):
        return mixer.forward(x, None, mixer.state(1), None, None, where)[0].double()

    base, moved, spread = run(at), run(at + 4096), run(at * 7)
    rms = base.square().mean().sqrt()
    assert (moved - base).abs().mean() <= 0.05 * rms < (spread - base).abs().mean()


@pytest.mark.parametrize("args", [["--mixer", "heads", "--heads", "2,8", "--rotate"], ["--mixer", "channels", "--heads", "1,4"],
                                  ["--heads", "2,4", "--rotate"]], ids=["heads", "channels", "delta"])
def test_example_runs(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "token_mixer.py"), "--layers", "2", "--width", "512",
                        "--prompts", "130,1,40", "--steps", "8", *args], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr
    assert "prompts:" in r.stdout and "decoding:" in r.stdout
