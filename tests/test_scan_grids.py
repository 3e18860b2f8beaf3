"""Sizes at the end of the grids of the selective scan of heads, on the host: what a grid of fewer than 2^32 threads does not
hold is unsupported, and a call that picks its form takes the other one."""
import pytest
import torch

import convolution_forward_amd as cf
from test_mixer_abi import lib  # noqa: F401
from test_scan_abi import HEADS

F32, BF = torch.float32, torch.bfloat16
HEADS_EACH = 8      # of as many groups, 16 columns each: one workgroup a group and segment number


def workgroups(seqs):
    """Of `seqs` single tokens by chunks: a number a sequence and one for every 64 tokens, each of eight workgroups."""
    return (seqs + seqs // 64) * HEADS_EACH


@pytest.mark.parametrize("dtype,code,threads", [(BF, cf.CONV_BF16, 512), (F32, cf.CONV_F32, 256)], ids=["bf16", "fp32"])
def test_chunk_grids_end(lib, dtype, code, threads):  # noqa: F811
    lo, hi = 1, 1 << 22         # fits, does not
    assert workgroups(lo) * threads < 1 << 32 <= workgroups(hi) * threads
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if workgroups(mid) * threads < 1 << 32 else (lo, mid)

    def space(n, variant):
        return cf.selective_scan_heads_workspace(n, n, HEADS_EACH, 16, HEADS_EACH, 16, dtype=dtype, variant=variant)
    assert space(lo, cf.VARIANT_TILED) >= 0
    assert space(hi, cf.VARIANT_TILED) == -1
    assert space(hi, cf.VARIANT_AUTO) == space(hi, cf.VARIANT_DIRECT) == 0
    call = {**HEADS, "T": hi, "n": hi, "num": hi, "H": HEADS_EACH, "P": 16, "G": HEADS_EACH, "N": 16, "ds": HEADS_EACH, "dt": code,
            "off": None, "slots": None, "variant": cf.VARIANT_TILED}
    assert lib.conv_selective_scan_heads_fwd(*call.values()) == cf.CONV_ERR_UNSUPPORTED


def test_longer_sequences_past_the_chunk_grid():
    """32769 sequences of seven tokens, 256 heads of their own group: long enough for chunks, of which there are too many."""
    n = 32769
    assert cf.selective_scan_heads_workspace(7 * n, n, 256, 16, 256, 16, variant=cf.VARIANT_TILED) == -1
    assert cf.selective_scan_heads_workspace(7 * n, n, 256, 16, 256, 16, variant=cf.VARIANT_AUTO) == 0
    assert cf.selective_scan_heads_workspace(7 * n, n, 256, 16, 256, 16, dtype=F32, variant=cf.VARIANT_TILED) >= 0
