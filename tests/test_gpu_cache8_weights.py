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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -118])
def test_values_far_from_one(kind, size):
    # every token's values are `size` (the open block's too); scores rise by less than a move of the references
    d, H, n = 64, 8, 4
    B = HEADS // H
    c = gb.cache8_alloc(B, 64 * (n + 1), H, d, kind)
    V = torch.full((B, 64 * n + 20, H, d), size, device="cuda").bfloat16()
    gb.cache8_append(c, torch.zeros_like(V), V, torch.zeros(B, dtype=torch.int32, device="cuda"))
    for j in range(n):
        c.k8.view(torch.uint8)[:, :, j, :, 0] = code(9 * j, kind)   # scores 0, 2.25, 4.5, 6.75 with queries of 2
    c.k_scale.fill_(1.0)
    lens = torch.full((B,), 64 * n + 19, dtype=torch.int32, device="cuda")
    O = gb.gated_sdpa_cache8(None, queries(B, 1, 4 * H, d, 2.0), c, lens, gate="none").double()
    # values through 8 bits: int8's amax is code 127 with a scale of two roundings, e4m3's within half a step of 2^-4;
    # one bf16 rounding; weights and their sum cancel but for 2^-10
    off = {"int8": 2.0 ** -22, "e4m3": 2.0 ** -4}[kind] + 2.0 ** -8 + 2.0 ** -10
    v = float(V[0, 0, 0, 0])
    assert float((O / v - 1).abs().max()) <= off


def check_heads(O, cache, Q, T, heads):
    """Some heads against the formula. A weight is rounded to fp16, 2^-11 of itself, or, below fp16's normal numbers,
    by 2^-25 at most, where the largest product of a weight and a value scale stands for 2^12 or more: 2^-37 of it for
    each unit of a code. Scores are exact products, below 2^6 in log2 units and rounded three times; every sum has at
    most T / 8 additions or steps, each off by 2^-23: together below 2^-14 of the sum of magnitudes. Then bf16."""
    B, Lq, Hq, d = Q.shape
    H, G = cache.H_kv, Hq // cache.H_kv
    assert T % 64 == 0 and T <= 4096
    for b, h in heads:
        k = (cache.k8[b, h].double() * cache.k_scale[b, h, :, None, None].double()).reshape(-1, d)[:T]
        codes = cache.v8[b, h].double().transpose(-1, -2).reshape(-1, d)[:T]
        scale = cache.v_scale[b, h].double().repeat_interleave(64)[:T]
        v = codes * scale[:, None]
        q = Q[b, 0, h * G:(h + 1) * G].double()
        w = torch.softmax(q @ k.T / math.sqrt(d), -1)
        ref, mag = w @ v, w @ v.abs()
        lost = 2.0 ** -37 * w.amax(-1, keepdim=True) * float(scale.max()) * codes.abs().sum(0)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14) * mag + lost
        err = (O[b, 0, h * G:(h + 1) * G].double() - ref).abs()
        assert bool((err <= tol).all()), (b, h, float((err / tol).max()), float((err.norm() / ref.norm())))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gap", [8, 12, 14, 16, 17, 19])
@pytest.mark.parametrize("G,at", [(4, 0), (4, 2047), (12, 100), (72, 0)])
def test_one_token_without_values_that_has_nearly_all_the_weight(kind, gap, G, at):
    # a first token (or another) `gap` above the others' scores, its values zero: the others' weights, e^-gap of its
    # own, are all of the output
    d, T, H = 64, 2048, 8
    heads = HEADS if G <= 8 else 640
    c = crafted(heads, H, T // 64, d, kind, 5)
    k = torch.randint(-1, 2, c.k8.shape[:-1], generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    c.k8[..., 0] = k.to(c.k8.dtype)
    c.k8.view(torch.uint8)[:, :, at // 64, at % 64, 0] = code(4 * gap, kind)
    c.v8.view(torch.uint8)[:, :, at // 64, :, at % 64] = 0
    Q = queries(heads // H, 1, G * H, d, 2.0)
    O = gb.gated_sdpa_cache8(None, Q, c, torch.full((heads // H,), T - 1, dtype=torch.int32, device="cuda"), gate="none")
    check_heads(O, c, Q, T, [(b, b % H) for b in range(0, heads // H, 17)])


@pytest.mark.parametrize("G", [4, 12])
def test_a_block_with_one_large_value(G):
    # one element 2^20 times the others', which its block's scale follows; every column keeps its bits
    d, T, H, heads = 64, 2048, 8, 1600 if G == 4 else 640
    c = crafted(heads, H, T // 64, d, "int8", 7)
    c.v8[:, :, 9] = 0
    c.v8[:, :, 9, 5, 11] = 127
    c.v_scale[:, :, 9] *= 2.0 ** 20
    Q = queries(heads // H, 1, G * H, d, 2.0)
    O = gb.gated_sdpa_cache8(None, Q, c, torch.full((heads // H,), T - 1, dtype=torch.int32, device="cuda"), gate="none")
    check_heads(O, c, Q, T, [(b, b % H) for b in range(0, heads // H, 17)])
