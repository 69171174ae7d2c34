"""Host-only checks of the operators around the attention: the rotary plan, and
refusals before any device work. No kernel is launched here."""
import ctypes
import math

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from ops_ref import frequencies


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gb.load()


@pytest.mark.parametrize("kw", [{}, dict(theta=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=2.5),
                                dict(scaling="parts", factor=8.0, orig_len=4096),
                                dict(scaling="parts", factor=40.0, orig_len=4096, beta_fast=16.0, beta_slow=2.0)])
@pytest.mark.parametrize("rd", [16, 64, 96, 128])
def test_rope_plan_holds_turns_per_position(rd, kw):
    r = gb.Rope(rd, **kw)
    w = frequencies(rd, **kw)
    for i in range(rd // 2):
        # a few roundings of the power and the division, 2^-53 each, and the 2^-64 grid
        assert abs(r.plan.turn[i] / 2.0 ** 64 - w[i] / (2 * math.pi)) <= 16 * 2.0 ** -53 * w[i] / (2 * math.pi) + 2.0 ** -64
    assert all(r.plan.turn[i] == 0 for i in range(rd // 2, 64))
    want = 0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "parts" else 1.0
    assert abs(r.plan.attn_scale - want) <= 2.0 ** -23


def test_rope_plan_refusals():
    for args, kw in [((0,), {}), ((24,), {}), ((144,), {}), ((64,), dict(theta=1.0)), ((64,), dict(theta=math.inf)),
                     ((64,), dict(scaling="linear", factor=0.5)), ((64,), dict(scaling="parts", factor=2.0, orig_len=0)),
                     ((64,), dict(scaling="parts", factor=2.0, orig_len=10, beta_fast=1.0, beta_slow=2.0)),
                     ((64,), dict(attn_scale=math.nan)), ((16,), dict(inv_freq=[math.inf] * 8))]:
        with pytest.raises(gb.GsdpaError) as e:
            gb.Rope(*args, **kw)
        assert e.value.status == gb.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        gb.Rope(32, inv_freq=[1.0] * 8)
    with pytest.raises(ValueError):
        gb.Rope(32, attn_scale=0.0)
    with pytest.raises(KeyError):
        gb.Rope(32, layout="other")


def rope_call(**kw):
    base = dict(Q=16, K=16, gamma_q=None, gamma_k=None, positions=None, Qo=16, Ko=16, ld_q=512, ld_k=256, ld_qo=512,
                ld_ko=256, B=2, L=3, H_q=4, H_kv=2, d_k=128, norm=1, eps=1e-6, rope=None, dtype=gb.BF16, stream=None)
    base.update(kw)
    return int(gb.load().gsdpa_qk_norm_rope(*base.values()))


def test_qk_norm_rope_validation_before_any_device_work():
    assert rope_call(B=-1) == gb.ERR_INVALID_ARG
    assert rope_call(H_kv=0) == gb.ERR_INVALID_ARG
    assert rope_call(dtype=2) == gb.ERR_INVALID_ARG
    assert rope_call(norm=2) == gb.ERR_INVALID_ARG
    assert rope_call(eps=-1.0) == gb.ERR_INVALID_ARG
    assert rope_call(eps=math.nan) == gb.ERR_INVALID_ARG
    assert rope_call(norm=0, gamma_k=16) == gb.ERR_INVALID_ARG
    assert rope_call(Q=None) == gb.ERR_INVALID_ARG
    assert rope_call(Ko=None) == gb.ERR_INVALID_ARG
    assert rope_call(ld_q=504) == gb.ERR_INVALID_ARG          # rows that overlap
    assert rope_call(ld_q=1024) == gb.ERR_INVALID_ARG         # in place with another row length
    assert rope_call(d_k=96) == gb.ERR_UNSUPPORTED
    assert rope_call(B=1 << 20, L=1 << 20) == gb.ERR_UNSUPPORTED
    assert rope_call(H_q=1 << 25) == gb.ERR_UNSUPPORTED
    assert rope_call(ld_k=260, Ko=32) == gb.ERR_ALIGNMENT     # a row that does not start on 16 bytes
    assert rope_call(Q=24) == gb.ERR_ALIGNMENT
    assert rope_call(gamma_q=24) == gb.ERR_ALIGNMENT
    assert rope_call(positions=2) == gb.ERR_ALIGNMENT
    assert rope_call(B=0) == gb.OK and rope_call(L=0) == gb.OK
    r = gb.Rope(128)
    r.plan.layout = 5
    assert rope_call(rope=r.ref) == gb.ERR_INVALID_ARG
    assert rope_call(rope=gb.Rope(128).ref, d_k=64, ld_q=256, ld_qo=256, ld_k=128, ld_ko=128) == gb.ERR_INVALID_ARG


def test_qk_norm_rope_bwd_workspace_and_validation():
    n = gb.qk_norm_rope_bwd_workspace_bytes(2, 2048, 128)
    assert n > 0 and n % (2 * 128 * 4) == 0
    assert gb.qk_norm_rope_bwd_workspace_bytes(2, 2048, 128, norm=False) == 0
    assert gb.qk_norm_rope_bwd_workspace_bytes(0, 2048, 128) == 0
    with pytest.raises(gb.GsdpaError):
        gb.qk_norm_rope_bwd_workspace_bytes(2, 2048, 96)
    f = gb.load().gsdpa_qk_norm_rope_bwd
    args = dict(Q=16, K=16, gamma_q=16, gamma_k=16, positions=None, dQo=16, dKo=16, dQ=16, dK=16, dgq=16, dgk=16, ld_q=512,
                ld_k=256, ld_dqo=512, ld_dko=256, ld_dq=512, ld_dk=256, B=2, L=3, H_q=4, H_kv=2, d_k=128, norm=1, eps=1e-6,
                rope=None, dtype=gb.BF16, ws=None, wsn=0, stream=None)

    def call(**kw):
        return int(f(*{**args, **kw}.values()))
    assert call(norm=0, gamma_q=None, gamma_k=None) == gb.ERR_INVALID_ARG      # gradients of a norm that is not there
    assert call(Q=None) == gb.ERR_INVALID_ARG
    assert call(dKo=None) == gb.ERR_INVALID_ARG
    assert call(ld_dq=1024) == gb.ERR_INVALID_ARG                               # in place with another row length
    assert call(dgq=8) == gb.ERR_ALIGNMENT
    assert call(dK=8) == gb.ERR_ALIGNMENT
    assert call(B=0) == gb.OK


def plan(**kw):
    base = dict(kind=0, B=2, H_kv=2, d_k=128, capacity=128, k8=16, v8=16, k_scale=4, v_scale=4, k_tail=16, v_tail=16)
    base.update(kw)
    return gb._Cache8Plan(*base.values())


BAD_CACHES = [(dict(kind=2), gb.ERR_INVALID_ARG), (dict(B=-1), gb.ERR_INVALID_ARG), (dict(H_kv=0), gb.ERR_INVALID_ARG),
              (dict(capacity=100), gb.ERR_INVALID_ARG), (dict(capacity=0), gb.ERR_INVALID_ARG),
              (dict(d_k=96), gb.ERR_UNSUPPORTED), (dict(k8=None), gb.ERR_INVALID_ARG), (dict(v_tail=None), gb.ERR_INVALID_ARG),
              (dict(v8=8), gb.ERR_ALIGNMENT), (dict(k_tail=24), gb.ERR_ALIGNMENT), (dict(v_scale=2), gb.ERR_ALIGNMENT)]


def append_call(p, **kw):
    base = dict(K=16, V=16, ld_k=256, ld_v=256, lens=4, n_new=None, L=3, stream=None)
    base.update(kw)
    return int(gb.load().gsdpa_cache8_append(None if p is None else ctypes.addressof(p), *base.values()))


def test_append_validation_before_any_device_work():
    for kw, st in BAD_CACHES:
        assert append_call(plan(**kw)) == st, kw
    assert append_call(None) == gb.ERR_INVALID_ARG
    assert append_call(plan(), K=None) == gb.ERR_INVALID_ARG
    assert append_call(plan(), lens=None) == gb.ERR_INVALID_ARG
    assert append_call(plan(), L=-1) == gb.ERR_INVALID_ARG
    assert append_call(plan(), ld_v=128) == gb.ERR_INVALID_ARG
    assert append_call(plan(), ld_v=260) == gb.ERR_ALIGNMENT
    assert append_call(plan(), V=8) == gb.ERR_ALIGNMENT
    assert append_call(plan(), n_new=2) == gb.ERR_ALIGNMENT
    assert append_call(plan(), L=0) == gb.OK
    assert append_call(plan(B=0)) == gb.OK


def attend_call(p, **kw):
    base = dict(X=16, Q=16, cache=None if p is None else ctypes.addressof(p), lens=4, n_new=None, W_g=16, O=16, L_q=1,
                d_model=64, H_q=8, gate_mode=2, workspace=None, workspace_bytes=0, stream=None)
    base.update(kw)
    return int(gb.load().gated_sdpa_cache8(*base.values()))


def test_attend_validation_before_any_device_work():
    for kw, st in BAD_CACHES:
        assert attend_call(plan(**kw)) == st, kw
    assert attend_call(None) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), H_q=7) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), gate_mode=3) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), d_model=0) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), X=None) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), Q=None) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), lens=None) == gb.ERR_INVALID_ARG
    assert attend_call(plan(), d_model=60) == gb.ERR_UNSUPPORTED
    assert attend_call(plan(), H_q=4, gate_mode=1) == gb.ERR_UNSUPPORTED        # headwise: H_q a multiple of 8
    assert attend_call(plan(), L_q=33) == gb.ERR_UNSUPPORTED                    # 4 x 33 query rows
    assert attend_call(plan(), O=8) == gb.ERR_ALIGNMENT
    assert attend_call(plan(), n_new=6) == gb.ERR_ALIGNMENT
    assert attend_call(plan(), L_q=0) == gb.OK
    assert attend_call(plan(B=0)) == gb.OK
    n = gb.load().gsdpa_cache8_workspace_bytes
    p = plan()
    a = ctypes.addressof(p)
    assert n(a, 1, 64, 8, 2) % 256 == 0 and n(a, 1, 64, 8, 2) > n(a, 1, 0, 8, 0) > 0
    assert n(a, 0, 64, 8, 2) == 0
    assert n(a, 33, 64, 8, 2) == ctypes.c_size_t(-1).value


def test_binding_rejects_host_tensors():
    Q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gb.qk_norm_rope(Q, Q)
    with pytest.raises(ValueError, match="CUDA"):
        gb.cache8_alloc(1, 64, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        gb.Cache8(torch.zeros(1, 1, 1, 64, 64), *[None] * 5)


def test_status_string():
    assert gb.status_string(gb.ERR_CACHE_RANGE) == "GSDPA_ERR_CACHE_RANGE"
