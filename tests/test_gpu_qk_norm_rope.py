"""Per-head norm with rotary positions, forward and backward, against the 64-bit
formula.

Tolerances. A result is a sum of two products of float32 factors: x, r (the
sum of d_k squares: at most 8 serial and 4 tree additions, then rsqrt within 2
units), gamma, t cos a (sincospif and the angle's conversion: each below 2^-22
absolute), so at most about 32 roundings of 2^-24 relative to the sum of the two
products' magnitudes; then one rounding to the output's type. The backward adds
the same count for the sum of h x and the second term: 64.
"""
import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from ops_ref import frequencies, half_step, norm_rope

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    gb.load()


def make(B, L, Hq, Hkv, d, dtype, seed, gamma=True):
    g = torch.Generator().manual_seed(seed)
    packed = torch.randn(B, L, (Hq + 2 * Hkv) * d, generator=g).to(dtype).cuda()
    Q = packed[..., :Hq * d].unflatten(-1, (Hq, d))
    K = packed[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    gq = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() if gamma else None
    gk = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() if gamma else None
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, L), generator=g).to(torch.int32)
    pos.view(-1)[::2] = torch.randint(0, 1_000_000, (B * L,), generator=g).to(torch.int32)[::2]
    return packed, Q, K, gq, gk, pos.cuda()


def rope_pair(rd, layout, **kw):
    if rd == 0:
        return None, None
    return gb.Rope(rd, layout=layout, **kw), frequencies(rd, **{k: v for k, v in kw.items() if k != "attn_scale"})


def check_forward(out, x, gamma, pos, w, layout, scale, norm, eps=1e-6):
    gd = None if gamma is None else gamma.double()
    ref = norm_rope(x.double(), gd, pos, w, layout, scale, norm, eps)
    y = norm_rope(x.double(), gd, pos, None, layout, scale, norm, eps).abs()
    mag = y.clone()
    if w is not None:   # the two members of a pair, by magnitude
        h = len(w)
        if layout == "half":
            both = y[..., :h] + y[..., h:2 * h]
            mag[..., :2 * h] = torch.cat((both, both), -1) * scale
        else:
            both = y[..., 0:2 * h:2] + y[..., 1:2 * h:2]
            mag[..., :2 * h] = torch.stack((both, both), -1).flatten(-2) * scale
    tol = half_step(out.dtype) * ref.abs() + 32 * U * mag
    bad = (out.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, worst {float(((out.double() - ref).abs() / (tol + 1e-300)).max()):.2f} x the tolerance"


SHAPES = [(1, 2, 131, 70, 64), (1, 1, 1, 1, 128), (2, 1, 8, 2, 64), (3, 7, 3, 1, 64), (2, 33, 16, 16, 128), (1, 300, 5, 2, 128)]
ROPES = [(0, "half", {}), (128, "half", {}), (64, "interleaved", {}), (16, "interleaved", dict(scaling="linear", factor=4.0)),
         (48, "half", dict(scaling="base", factor=3.0, theta=500000.0)),
         (64, "half", dict(scaling="parts", factor=8.0, orig_len=4096))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[1]}{r[0]}{r[2].get('scaling', '')}")
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, rope, norm, dtype):
    B, L, Hq, Hkv, d = shape
    rd = min(rope[0], d)
    _, Q, K, gq, gk, pos = make(B, L, Hq, Hkv, d, dtype, 1, gamma=norm)
    plan, w = rope_pair(rd, rope[1], **rope[2])
    scale = 0.1 * torch.tensor(8.0).double().log().item() + 1 if rope[2].get("scaling") == "parts" else 1.0
    q, k = gb.qk_norm_rope(Q, K, gamma_q=gq, gamma_k=gk, norm=norm, rope=plan, positions=pos)
    assert q.is_contiguous() and q.shape == Q.shape and k.shape == K.shape
    check_forward(q, Q, gq, pos, w, rope[1], scale, norm)
    check_forward(k, K, gk, pos, w, rope[1], scale, norm)


def test_forward_many_tokens_default_positions():
    # one warp to a token, several heads to a warp, positions 0 .. L - 1 of every sequence
    B, L, Hq, Hkv, d = 2, 3001, 9, 3, 128
    _, Q, K, gq, gk, _ = make(B, L, Hq, Hkv, d, torch.bfloat16, 2)
    plan, w = rope_pair(128, "half")
    q, k = gb.qk_norm_rope(Q, K, gamma_q=gq, gamma_k=gk, rope=plan)
    pos = torch.arange(L, device="cuda").expand(B, L)
    check_forward(q, Q, gq, pos, w, "half", 1.0, True)
    check_forward(k, K, gk, pos, w, "half", 1.0, True)


def test_frequencies_of_the_callers_own_and_scale():
    w = [0.5 / (i + 1) for i in range(16)]
    w[3], w[4] = 7.0, -0.25   # more than a turn per position, and backwards
    _, Q, K, _, _, pos = make(2, 5, 4, 2, 64, torch.float32, 3, gamma=False)
    pos = pos.clamp(-100_000, 100_000)
    plan = gb.Rope(32, layout="half", inv_freq=w, attn_scale=0.5)
    q, _ = gb.qk_norm_rope(Q, K, rope=plan, positions=pos)
    check_forward(q, Q, None, pos, w, "half", 0.5, True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_on_a_packed_projection_leaves_the_rest(layout, dtype):
    B, L, Hq, Hkv, d = 2, 37, 8, 4, 128
    packed, Q, K, gq, gk, pos = make(B, L, Hq, Hkv, d, dtype, 4)
    plan, _ = rope_pair(96, layout)
    q, k = gb.qk_norm_rope(Q, K, gamma_q=gq, gamma_k=gk, rope=plan, positions=pos)
    before = packed.clone()
    out = gb.qk_norm_rope(Q, K, gamma_q=gq, gamma_k=gk, rope=plan, positions=pos, out_q=Q, out_k=K)
    assert out[0].data_ptr() == Q.data_ptr()
    assert torch.equal(Q, q) and torch.equal(K, k)
    assert torch.equal(packed[..., (Hq + Hkv) * d:], before[..., (Hq + Hkv) * d:])   # V


def test_rows_of_zeros_and_special_values():
    Q = torch.zeros(1, 4, 2, 64, device="cuda")
    Q[0, 1, 0, 3] = float("nan")
    Q[0, 2, 1, 5] = float("inf")
    K = torch.zeros(1, 4, 1, 64, device="cuda")
    q, k = gb.qk_norm_rope(Q, K, rope=gb.Rope(64))
    assert torch.equal(k, torch.zeros_like(k))
    bad = torch.isnan(q).any(-1)[0]
    want = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    want[1, 0] = want[2, 1] = True
    assert torch.equal(bad, want)           # and no other row


# ---------------------------------------------------------------- backward
def reference_grads(x, gamma, dz, pos, w, layout, scale, norm, eps=1e-6):
    x64 = x.double().detach().requires_grad_()
    g64 = (torch.ones(x.shape[-1], device=x.device) if gamma is None else gamma).double().detach().requires_grad_()
    norm_rope(x64, g64 if norm else None, pos, w, layout, scale, norm, eps).backward(dz.double())
    return x64.grad, g64.grad


def grad_magnitudes(x, gamma, dz, w, layout, scale, norm, eps=1e-6):
    """Magnitudes that the roundings of dx and of dgamma's terms are relative to."""
    a = dz.double().abs()
    if w is not None:
        h = len(w)
        if layout == "half":
            both = (a[..., :h] + a[..., h:2 * h]) * scale
            a = torch.cat((both, both, a[..., 2 * h:]), -1)
        else:
            both = (a[..., 0:2 * h:2] + a[..., 1:2 * h:2]) * scale
            a = torch.cat((torch.stack((both, both), -1).flatten(-2), a[..., 2 * h:]), -1)
    if not norm:
        return a, None
    r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + eps)
    xh = x.double().abs() * r
    hh = a * (1 if gamma is None else gamma.double().abs())
    return r * (hh + xh * (hh * xh).mean(-1, keepdim=True)), (a * xh).sum((0, 1, 2))


def check_backward(out, name, x, gamma, dz, pos, w, layout, scale, norm):
    dx, dg = reference_grads(x, gamma, dz, pos, w, layout, scale, norm)
    mx, mg = grad_magnitudes(x, gamma, dz, w, layout, scale, norm)
    got = out["d" + name]
    tol = half_step(got.dtype) * dx.abs() + 64 * U * mx
    assert bool(((got.double() - dx).abs() <= tol).all())
    if norm:
        got = out["dgamma_" + name.lower()]
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        # (a thread adds at most all rows one after another; each term has 32 roundings)
        tol = half_step(got.dtype) * dg.abs() + (32 + rows) * U * mg
        assert bool(((got.double() - dg).abs() <= tol).all())
    else:
        assert "dgamma_" + name.lower() not in out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[1]}{r[0]}{r[2].get('scaling', '')}")
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, rope, norm, dtype):
    B, L, Hq, Hkv, d = shape
    rd = min(rope[0], d)
    _, Q, K, gq, gk, pos = make(B, L, Hq, Hkv, d, dtype, 5, gamma=norm)
    g = torch.Generator().manual_seed(6)
    dQ = torch.randn(B, L, Hq, d, generator=g).to(dtype).cuda()
    dK = torch.randn(B, L, Hkv, d, generator=g).to(dtype).cuda()
    plan, w = rope_pair(rd, rope[1], **rope[2])
    scale = 0.1 * torch.tensor(8.0).double().log().item() + 1 if rope[2].get("scaling") == "parts" else 1.0
    out = gb.qk_norm_rope_bwd(Q, K, dQ, dK, gamma_q=gq, gamma_k=gk, norm=norm, rope=plan, positions=pos)
    check_backward(out, "Q", Q, gq, dQ, pos, w, rope[1], scale, norm)
    check_backward(out, "K", K, gk, dK, pos, w, rope[1], scale, norm)


def test_backward_many_rows_without_gamma_in_place_and_repeated():
    B, L, Hq, Hkv, d = 2, 4000, 4, 2, 64
    _, Q, K, _, _, _ = make(B, L, Hq, Hkv, d, torch.float32, 7, gamma=False)
    g = torch.Generator().manual_seed(8)
    dQ, dK = torch.randn(B, L, Hq, d, generator=g).cuda(), torch.randn(B, L, Hkv, d, generator=g).cuda()
    plan, w = rope_pair(64, "interleaved")
    pos = torch.arange(L, device="cuda").expand(B, L)
    out = gb.qk_norm_rope_bwd(Q, K, dQ, dK, rope=plan)
    check_backward(out, "Q", Q, None, dQ, pos, w, "interleaved", 1.0, True)
    check_backward(out, "K", K, None, dK, pos, w, "interleaved", 1.0, True)
    again = gb.qk_norm_rope_bwd(Q, K, dQ, dK, rope=plan)
    assert all(torch.equal(out[n], again[n]) for n in out)          # a fixed order of additions
    here = gb.qk_norm_rope_bwd(Q, K, dQ, dK, rope=plan, out_dq=dQ, out_dk=dK)
    assert here["dQ"].data_ptr() == dQ.data_ptr()
    assert torch.equal(dQ, out["dQ"]) and torch.equal(dK, out["dK"])


def test_backward_against_differences():
    # the quotient of the 64-bit forward along a random direction: with step 1e-5 it
    # is off by about 1e-10 (third derivatives of order one) + 1e-16 / 1e-5
    B, L, Hq, Hkv, d = 1, 3, 2, 1, 64
    _, Q, K, gq, gk, pos = make(B, L, Hq, Hkv, d, torch.float32, 9)
    g = torch.Generator().manual_seed(10)
    dQ, dK = torch.randn(B, L, Hq, d, generator=g).cuda(), torch.randn(B, L, Hkv, d, generator=g).cuda()
    plan, w = rope_pair(32, "half")
    out = gb.qk_norm_rope_bwd(Q, K, dQ, dK, gamma_q=gq, gamma_k=gk, rope=plan, positions=pos)
    h = 1e-5
    for seed in range(4):
        v = torch.randn(Q.shape, generator=torch.Generator().manual_seed(20 + seed)).double().cuda()
        vg = torch.randn(d, generator=torch.Generator().manual_seed(30 + seed)).double().cuda()

        def f(s):
            y = norm_rope(Q.double() + s * v, gq.double() + s * vg, pos, w, "half")
            return float((y * dQ.double()).sum())
        quotient = (f(h) - f(-h)) / (2 * h)
        got = float((out["dQ"].double() * v).sum() + (out["dgamma_q"].double() * vg).sum())
        mx, mg = grad_magnitudes(Q, gq, dQ, w, "half", 1.0, True)
        # the kernel's own roundings along v, and the quotient's error relative to the sum of magnitudes
        tol = 66 * U * float((mx * v.abs()).sum() + (mg * vg.abs()).sum())
        assert abs(got - quotient) <= tol


# ---------------------------------------------------------------- streams, graphs, refusals
def test_captured_and_replayed_beside_an_eager_call():
    B, L, Hq, Hkv, d = 2, 9, 8, 2, 128
    _, Q, K, gq, gk, pos = make(B, L, Hq, Hkv, d, torch.bfloat16, 11)
    plan = gb.Rope(128)
    kw = dict(gamma_q=gq, gamma_k=gk, rope=plan, positions=pos)
    q0, k0 = gb.qk_norm_rope(Q, K, **kw)
    g0 = gb.qk_norm_rope_bwd(Q, K, q0, k0, **kw)
    outs = [torch.empty_like(q0), torch.empty_like(k0)]
    ws = torch.empty(gb.qk_norm_rope_bwd_workspace_bytes(B, L, d), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gb.qk_norm_rope(Q, K, out_q=outs[0], out_k=outs[1], **kw)
        g1 = gb.qk_norm_rope_bwd(Q, K, outs[0], outs[1], workspace=ws, **kw)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], q0) and torch.equal(outs[1], k0)
    assert all(torch.equal(g0[n], g1[n]) for n in g0)


def test_on_another_stream_after_the_current_one():
    # the outputs belong to the stream that the call ran on
    _, Q, K, gq, gk, pos = make(2, 2000, 8, 2, 128, torch.bfloat16, 12)
    kw = dict(gamma_q=gq, gamma_k=gk, rope=gb.Rope(64), positions=pos)
    want = gb.qk_norm_rope(Q, K, **kw)
    grads = gb.qk_norm_rope_bwd(Q, K, *want, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        q, k = gb.qk_norm_rope(Q, K, stream=side, **kw)
        got = gb.qk_norm_rope_bwd(Q, K, q, k, stream=side, **kw)
        side.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert all(torch.equal(got[n], grads[n]) for n in grads)


def test_refusals():
    Q, K = torch.zeros(2, 3, 4, 64, device="cuda"), torch.zeros(2, 3, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q, K[:, :2])
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q.transpose(2, 3), K)                          # not heads of contiguous columns
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q, K, positions=torch.zeros(2, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q, K, positions=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q, K, gamma_q=torch.ones(64, device="cuda").bfloat16())
    with pytest.raises(TypeError):
        gb.qk_norm_rope(Q.half(), K.half())
    with pytest.raises(ValueError):
        gb.qk_norm_rope(Q[:, :1].expand(2, 3, 4, 64), K)               # the same row for every token
    with pytest.raises(gb.GsdpaError) as e:
        gb.qk_norm_rope(Q, K, rope=gb.Rope(128))                       # wider than the head
    assert e.value.status == gb.ERR_INVALID_ARG
    with pytest.raises(gb.GsdpaError) as e:
        gb.qk_norm_rope(Q, K, norm=False, gamma_q=torch.ones(64, device="cuda"))
    assert e.value.status == gb.ERR_INVALID_ARG
    with pytest.raises(gb.GsdpaError) as e:
        gb.qk_norm_rope_bwd(Q, K, Q, K, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gb.ERR_WORKSPACE
    odd = torch.zeros(2 * 3 * 4 * 64 + 1, device="cuda")[1:].view(2, 3, 4, 64)
    with pytest.raises(gb.GsdpaError) as e:
        gb.qk_norm_rope(odd, K)
    assert e.value.status == gb.ERR_ALIGNMENT
    empty = gb.qk_norm_rope_bwd(Q[:, :0], K[:, :0], Q[:, :0], K[:, :0])
    assert not bool(empty["dgamma_q"].any()) and empty["dQ"].shape == (2, 0, 4, 64)
