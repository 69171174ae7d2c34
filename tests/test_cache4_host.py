"""Host-only checks of the paged 4-bit cache: refusals before any device work, the
handle, and the references that the GPU tests use. No kernel is launched here."""
import copy
import ctypes
import pickle

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
import cache4_ref as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gb.load()


def plan(**kw):
    base = dict(kind=0, n_pages=4, H_kv=2, d_k=128, k_exp=0, v_exp=0, pool=16)
    base.update(kw)
    return gb._Cache4Plan(*base.values())


BAD_CACHES = [(dict(kind=2), gb.ERR_INVALID_ARG), (dict(kind=-1), gb.ERR_INVALID_ARG), (dict(n_pages=0), gb.ERR_INVALID_ARG),
              (dict(H_kv=0), gb.ERR_INVALID_ARG), (dict(d_k=96), gb.ERR_UNSUPPORTED), (dict(k_exp=65), gb.ERR_INVALID_ARG),
              (dict(v_exp=-65), gb.ERR_INVALID_ARG), (dict(pool=None), gb.ERR_INVALID_ARG), (dict(pool=24), gb.ERR_ALIGNMENT)]


def address(p):
    return None if p is None else ctypes.addressof(p)


def pages_call(**kw):
    base = dict(lens=4, keep=None, n_new=4, table=4, free_pages=4, n_free=4, n_free_out=4, cu=4, granted=4, slots=8,
                positions=4, B=2, max_pages=3, n_pages=4, n_rows=5, stream=None)
    base.update(kw)
    return int(gb.load().gsdpa_pages_step(*base.values()))


def test_pages_step_validation_before_any_device_work():
    for name in ("lens", "n_new", "table", "free_pages", "n_free", "n_free_out", "cu", "granted", "slots"):
        assert pages_call(**{name: None}) == gb.ERR_INVALID_ARG, name
    for name in ("B", "n_rows"):
        assert pages_call(**{name: -1}) == gb.ERR_INVALID_ARG
    for name in ("max_pages", "n_pages"):
        assert pages_call(**{name: 0}) == gb.ERR_INVALID_ARG
    assert pages_call(B=8193) == gb.ERR_UNSUPPORTED
    assert pages_call(max_pages=1 << 25) == gb.ERR_UNSUPPORTED          # more than 2^31 tokens
    assert pages_call(n_rows=0x7fffffff) == gb.ERR_UNSUPPORTED
    for name in ("lens", "keep", "n_new", "table", "free_pages", "n_free", "n_free_out", "cu", "granted", "positions"):
        assert pages_call(**{name: 6}) == gb.ERR_ALIGNMENT, name
    assert pages_call(slots=4) == gb.ERR_ALIGNMENT


@pytest.mark.parametrize("name", ["gsdpa_cache4_append", "gsdpa_cache4_read"])
def test_rows_validation_before_any_device_work(name):
    def call(p, **kw):
        v = dict(K=16, V=16, ld_k=256, ld_v=256, slots=8, n_rows=3)
        v.update(kw)
        rows = (v["K"], v["V"], v["ld_k"], v["ld_v"])
        args = (*rows, v["slots"]) if name.endswith("append") else (v["slots"], *rows)
        return int(getattr(gb.load(), name)(address(p), *args, v["n_rows"], None))
    for kw, st in BAD_CACHES:
        assert call(plan(**kw)) == st, kw
    assert call(None) == gb.ERR_INVALID_ARG
    for arg in ("K", "V", "slots"):
        assert call(plan(), **{arg: None}) == gb.ERR_INVALID_ARG
    assert call(plan(), n_rows=-1) == gb.ERR_INVALID_ARG
    assert call(plan(), ld_v=248) == gb.ERR_INVALID_ARG                 # rows that overlap
    assert call(plan(), ld_k=260) == gb.ERR_ALIGNMENT
    assert call(plan(), K=8) == gb.ERR_ALIGNMENT
    assert call(plan(), slots=4) == gb.ERR_ALIGNMENT
    assert call(plan(H_kv=65536), ld_k=1 << 23, ld_v=1 << 23) == gb.ERR_UNSUPPORTED
    assert call(plan(), n_rows=0) == gb.OK


def attend_call(p, **kw):
    base = dict(X=16, Q=16, cache=address(p), table=4, lens=4, cu=4, n_new=None, W_g=16, O=16, B=2, max_pages=3, n_rows=2,
                max_new=1, d_model=64, H_q=8, gate_mode=2, workspace=None, workspace_bytes=0, stream=None)
    base.update(kw)
    return int(gb.load().gated_sdpa_cache4(*base.values()))


def test_attend_validation_before_any_device_work():
    for kw, st in BAD_CACHES:
        assert attend_call(plan(**kw)) == st, kw
    assert attend_call(None) == gb.ERR_INVALID_ARG
    for arg in ("X", "Q", "table", "lens", "cu", "W_g", "O"):
        assert attend_call(plan(), **{arg: None}) == gb.ERR_INVALID_ARG, arg
    for bad in (dict(B=-1), dict(n_rows=-1), dict(max_new=0), dict(max_pages=0), dict(H_q=7), dict(H_q=0), dict(gate_mode=3),
                dict(gate_mode=-1), dict(d_model=0)):
        assert attend_call(plan(), **bad) == gb.ERR_INVALID_ARG, bad
    for bad in (dict(d_model=60), dict(H_q=4, gate_mode=1), dict(max_new=33), dict(max_pages=1 << 25),
                dict(B=1 << 20, max_pages=1 << 20), dict(n_rows=1 << 29)):
        assert attend_call(plan(), **bad) == gb.ERR_UNSUPPORTED, bad
    for bad in (dict(Q=8), dict(O=24), dict(X=8), dict(W_g=2), dict(table=2), dict(lens=6), dict(cu=2), dict(n_new=6)):
        assert attend_call(plan(), **bad) == gb.ERR_ALIGNMENT, bad
    assert attend_call(plan(), n_rows=0) == gb.OK
    n = gb.load().gsdpa_cache4_workspace_bytes
    p = plan()
    assert n(address(p), 2, 3, 2, 1, 64, 8, 2) > n(address(p), 2, 3, 2, 1, 0, 8, 0) > 0
    assert n(address(p), 0, 3, 2, 1, 0, 8, 0) == 0
    assert n(address(p), 2, 3, 2, 33, 0, 8, 0) == ctypes.c_size_t(-1).value


@pytest.fixture
def on_the_host(monkeypatch):
    """Cache4 over host memory: no kernel sees it."""
    monkeypatch.setattr(gb, "_expect", lambda *a: None)


def test_handle_checks(on_the_host):
    pool = torch.zeros(3, 2, 72 * 64, dtype=torch.uint8)
    c = gb.Cache4(pool, "int4", k_exp=-3, v_exp=2)
    assert (c.plan.kind, c.plan.n_pages, c.plan.H_kv, c.plan.d_k, c.plan.k_exp, c.plan.v_exp) == (0, 3, 2, 64, -3, 2)
    with pytest.raises(TypeError):
        gb.Cache4(pool.int())
    for bad in (dict(kind="int8"), dict(k_exp=65), dict(v_exp=0.5)):
        with pytest.raises(ValueError):
            gb.Cache4(pool, **bad)
    with pytest.raises(ValueError):
        gb.Cache4(pool[..., :100])
    with pytest.raises(ValueError):
        gb.Cache4(pool[0])


def test_a_copied_handle_is_over_its_own_pool(on_the_host):
    c = gb.Cache4(torch.zeros(2, 1, 72 * 128, dtype=torch.uint8), "e2m1", k_exp=-4, v_exp=1)
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert other.plan.pool == other.pool.data_ptr() != c.pool.data_ptr()
        assert other.ref == ctypes.addressof(other.plan) != c.ref
        assert (other.kind, other.plan.k_exp, other.plan.v_exp) == ("e2m1", -4, 1)
    assert copy.copy(c).plan.pool == c.pool.data_ptr()


def test_binding_rejects_host_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        gb.cache4_alloc(1, 1, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gb.pages_step(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1], 2)
    with pytest.raises(ValueError):
        gb.pages_step(i, i, i, i, i[:1], 2)


# ---------------------------------------------------------------- the references
@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_page_has_a_place_for_everything_and_no_more(d, kind):
    k, v, ks, vs = ref.places(d, kind)
    used = torch.zeros(72 * d, 2, dtype=torch.int64)
    for x in (k, v):
        used.view(-1).index_add_(0, (2 * x[..., 0] + x[..., 1] // 4).flatten(), torch.ones(x[..., 0].numel(), dtype=torch.int64))
    for x in (ks, vs):
        used.index_add_(0, x.flatten(), torch.ones(x.numel(), 2, dtype=torch.int64))
    assert bool((used == 1).all())
    # a token's bytes are its own: no byte has codes of two
    for x in (k, v):
        owner = torch.full((72 * d,), -1)
        for n in range(64):
            assert bool((owner[x[n, :, 0]] == -1).all())
            owner[x[n, :, 0]] = n


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
def test_reference_codes_by_hand(kind):
    x = torch.zeros(16, dtype=torch.float64)
    top = ref.TOP[kind]
    x[0], x[1], x[2], x[3], x[4] = top, 2.5, -3.5, 0.25, -1.75      # scale 1; ties go to even codes
    codes, scale = ref.quantise(x, kind, 0)
    assert float(scale) == 1.0
    assert codes[:5].tolist() == ([7.0, 2.0, -4.0, 0.0, -2.0] if kind == "int4" else [6.0, 2.0, -4.0, 0.0, -2.0])
    codes, scale = ref.quantise(x * 1024, kind, 10)
    assert float(scale) == 1.0 and float(codes[2]) == -4.0
    codes, scale = ref.quantise(x * 1000, kind, 0)                  # cut off at 448
    assert float(scale) == 448.0 and float(codes[0]) == top
    codes, scale = ref.quantise(x * 2.0 ** -11, kind, 0)            # under half of the least scale
    assert float(scale) == 0.0 and not bool(codes.any())
    x[5] = float("inf")
    codes, scale = ref.quantise(x, kind, 0)
    assert bool(scale.isnan()) and not bool(codes.any())


def test_reference_plan_by_hand():
    # 100 -> 40 tokens gives page 9 back; then 30 more need one, and 65 new ones two: the stack has 9 on top
    cu, granted, slots, positions, left, table, _ = ref.plan([100, 0, 64], [30, 65, 1], [[8, 9], [-1, -1], [3, -1]], [5, 6, 7], 3,
                                                             98, 2, keep=[40, 0, 64])
    assert cu == [0, 30, 95, 96] and granted == [30, 65, 1] and left == 0
    assert table == [[8, 9], [7, 6], [3, 5]]
    assert slots[0] == 8 * 64 + 40 and slots[24] == 9 * 64 and slots[30] == 7 * 64 and slots[95] == 5 * 64 and slots[96:] == [-1, -1]
    assert positions[:2] == [40, 41] and positions[95] == 64 and positions[96:] == [0, 0]
