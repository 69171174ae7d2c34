"""The attention over the 8-bit cache where one token or block outweighs the others:
caches written by hand, so many heads that each is one team's from end to end.

The queries have one element that is not zero, a power of two, so that every score is
one exact product: q code scale / sqrt(d). Scores then follow the first column of the
keys' codes alone.
"""
import math

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
KINDS = ["int8", "e4m3"]
HEADS = 1600   # more than there are teams of warps: no head of a few tiles is cut into single ones


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    gb.load()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert gb.check_device_error() == gb.OK


def crafted(heads, H, n, d, kind, seed):
    """A cache of n blocks for each of `heads` (sequence, K/V head) pairs: keys' codes zero, key scales
    one, values of random codes with scales that make them about one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = heads // H
    c = gb.cache8_alloc(B, 64 * n, H, d, kind)
    v = torch.randn(c.v8.shape, generator=g, device="cuda")
    if kind == "int8":
        c.v8.copy_((v * 40).round().clamp(-127, 127).to(torch.int8))
        c.v_scale.copy_((0.7 + 0.6 * torch.rand(c.v_scale.shape, generator=g, device="cuda")) / 40)
    else:
        c.v8.copy_((v * 64).clamp(-448, 448).to(torch.float8_e4m3fn))
        c.v_scale.fill_(2.0 ** -6)
    c.k8.view(torch.uint8).zero_()
    c.k_scale.fill_(1.0)
    c.k_tail.zero_()
    c.v_tail.copy_(torch.randn(c.v_tail.shape, generator=g, device="cuda"))
    return c


def code(x, kind):
    return torch.tensor(float(x), device="cuda").to(torch.int8 if kind == "int8" else torch.float8_e4m3fn).view(torch.uint8)


def queries(B, Lq, Hq, d, size):
    Q = torch.zeros(B, Lq, Hq, d, device="cuda", dtype=torch.bfloat16)
    Q[..., 0] = size
    return Q


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,rest,where", [(1, 0, 0), (4, 0, 1), (4, 9, 0), (12, 0, 0), (12, 9, 1), (72, 0, 0)])
def test_a_block_without_values_that_has_all_the_weight(kind, G, rest, where):
    # keys of one block 120 above the others' scores (e^-120 of its weights), its values zero with the scale zero
    # that the append gives such a block, or next to nothing: the output is zero, whatever comes after it
    d, n, H = 64, 4, 8
    heads = HEADS if G <= 8 else 640
    c = crafted(heads, H, n + (1 if rest else 0), d, kind, 1)
    c.k8.view(torch.uint8)[:, :, where, :, 0] = code(60, kind)
    for scale in (0.0, 2.0 ** -115):
        c.v_scale[:, :, where] = scale
        if scale == 0.0:
            c.v8.view(torch.uint8)[:, :, where] = 0
        else:
            c.v8.view(torch.uint8)[:, :, where] = code(3, kind)
        B = heads // H
        lens = torch.full((B,), 64 * n + rest - 1, dtype=torch.int32, device="cuda")
        O = gb.gated_sdpa_cache8(None, queries(B, 1, G * H, d, 16.0), c, lens, gate="none")
        assert bool(torch.isfinite(O).all()), f"{int((~torch.isfinite(O)).sum())} of {O.numel()}"
        # (the other blocks have about e^-120 = 2^-173 of the weight and values below 2^3)
        assert float((O.double() - 3 * scale).abs().max()) <= 2.0 ** -8 * 3 * scale + 2.0 ** -120
