"""The token-mixer operators together, as examples/token_mixer.py runs them."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import token_mixer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().to(DEV)


@pytest.mark.parametrize("qtype", [torch.int8, torch.float8_e4m3fn])
def test_prompt_then_single_tokens(qtype):
    """A prompt in one call (chunks, tiles) equals the same prompt cut, its last tokens one by one (recurrent, few rows).

    Sums in another order turn a bf16 rounding now and then: of o, by the delta rule's 1e-7, and in e4m3 of the
    projection too (int8 sums are exact). At worst that moves a row's scale by 2^-8, and with it 8-bit values by a step
    each: 1/127 of the row's largest (1/16 of the value itself in e4m3), some 3 times the row's RMS. Such steps at random
    in all K places leave about 2 % of the outputs' RMS, and 5 deviations of it are 0.1. States hold such values (2^-8
    each, so 2^-6 with room), or in int8 the same ones.
    """
    lens, last = [150, 70, 1, 0, 33], [6, 6, 1, 0, 6]
    n = len(lens)
    layer = token_mixer.TokenMixer(256, 2, 4, 128, 64, qtype, seed=3)
    x = torch.randn(sum(lens), 256, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    slots = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32, device=DEV)
    whole, cut = layer.state(n), layer.state(n)
    want, _ = layer.forward(x, None, whole, offsets(lens), slots)
    rows = list(torch.arange(sum(lens), device=DEV).split(lens))
    head = [a - b for a, b in zip(lens, last)]
    got = torch.zeros_like(want)

    def step(index, counts):
        got[index], _ = layer.forward(x[index], None, cut, offsets(counts), slots)

    step(torch.cat([r[:m] for r, m in zip(rows, head)]), head)
    for t in range(max(last)):
        counts = [int(t < b) for b in last]
        step(torch.cat([r[m + t:m + t + c] for r, m, c in zip(rows, head, counts)]), counts)
    rms = want.double().square().mean().sqrt()
    assert torch.isfinite(want).all() and rms > 0
    assert ((got.double() - want.double()).abs().max() / rms).item() <= 0.1
    if qtype == torch.int8:
        assert torch.equal(whole[0], cut[0])    # rows of the convolution's input
    for a, b, part in zip(cut, whole, (2 ** -6, 1e-5 if qtype == torch.int8 else 2 ** -6)):
        assert (a.float() - b.float()).abs().max().item() <= part * b.float().abs().max().item()


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "token_mixer.py"), "--layers", "2", "--width", "512",
                        "--heads", "2,4", "--prompts", "130,1,40", "--steps", "8"], capture_output=True, text=True,
                       timeout=110)
    assert r.returncode == 0, r.stderr
    assert "prompts:" in r.stdout and "decoding:" in r.stdout
