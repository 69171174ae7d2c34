"""The paged 4-bit cache's append and reading back: bytes, codes and scales exactly as
the formulas say, whatever the order of the slots."""
import math

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from cache4_ref import CODES, GROUP, PAGE, TOP, codes_and_scales, held, places, quantise

pytestmark = pytest.mark.gpu
KINDS = ["int4", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    gb.load()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert gb.check_device_error() == gb.OK


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def slots_of(*v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def filled(n_pages, H, d, kind, byte=0xA5, **kw):
    c = gb.cache4_alloc(n_pages, H, d, kind, **kw)
    c.pool.fill_(byte)
    return c


def check(cache, before, K, V, slots):
    """The tokens at slots are K's and V's rows to the last bit, all others' bytes as they were."""
    live = [(i, s) for i, s in enumerate(slots.tolist()) if s >= 0]
    if live:
        rows, at = [i for i, _ in live], [s for _, s in live]
        k, v, ks, vs = (x.cpu() for x in codes_and_scales(cache.pool, at, cache.kind))
        for x, codes, scales, exp in ((K, k, ks, cache.k_exp), (V, v, vs, cache.v_exp)):
            want, scale = quantise(x.double().cpu()[rows], cache.kind, exp)
            assert torch.equal(codes, want)
            assert torch.equal(scales.nan_to_num(nan=-1.0), scale.nan_to_num(nan=-1.0))
    others = sorted(set(range(cache.n_pages * PAGE)) - {s for _, s in live})
    if others:
        for a, b in zip(codes_and_scales(cache.pool, others, cache.kind), codes_and_scales(before, others, cache.kind)):
            assert torch.equal(a.nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0))


ORDERS = {
    "one": [70],
    "last": [5 * 64 - 1],
    "tile": list(range(64, 80)),
    "pages": list(range(64, 256)),
    "odd": list(range(69, 69 + 131)),
    "backwards": list(range(200, 60, -1)),
    "scattered": [(37 * i + 11) % 320 for i in range(100)],
    "holes": [s if s % 3 else -1 for s in range(100, 200)],
    "none": [-1, -1, -5],
    "pieces": list(range(3, 40)) + [-1] * 9 + list(range(250, 300)) + list(range(130, 150)),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,d", [(1, 64), (3, 128), (2, 64), (5, 128)])
@pytest.mark.parametrize("order", list(ORDERS))
def test_append_writes_exactly_the_formula(order, H, d, kind):
    slots = slots_of(*ORDERS[order])
    N = len(slots)
    cache = filled(5, H, d, kind, k_exp=-5, v_exp=-3)
    before = cache.pool.clone()
    K, V = randn(1, N, H, d) * 2.5, randn(2, N, H, d)
    gb.cache4_append(cache, K, V, slots)
    check(cache, before, K, V, slots)


@pytest.mark.parametrize("kind", KINDS)
def test_values_where_rounding_is_decided(kind):
    # every scale's significand with every tie between codes, scales on ties, tiny and huge magnitudes, zeros of
    # both signs, powers of two
    d, rows = 128, []
    half_ways = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] if kind == "e2m1" else [k + 0.5 for k in range(7)]
    for m in range(8, 16):
        for e in (-9, -3, 0, 4):
            row = torch.zeros(d)
            row[0::16] = TOP[kind] * m * 2.0 ** e
            for i, h in enumerate(half_ways):
                row[1 + i::16] = h * m * 2.0 ** e * (-1.0 if (i + m) % 2 else 1.0)
            row[9::16] = -0.0
            rows.append(row)
    for mid in range(17, 32, 2):                                   # half way between two scales
        row = torch.zeros(d)
        row[3::16] = TOP[kind] * mid / 4
        row[4::16] = -mid / 8
        rows.append(row)
    for e in (-133, -126, -60, -20, -12, -11, -10, -9, 8, 11, 12, 60, 127):
        row = torch.linspace(-1, 1, d) * 2.0 ** e
        rows.append(row)
    K = torch.stack(rows)[:, None].bfloat16().cuda()
    V = -K.flip(0).contiguous()
    slots = torch.arange(len(rows), device="cuda")
    for exp in (0, -4, 7, -64, 64):
        cache = filled(2, 1, d, kind, k_exp=exp, v_exp=-exp)
        before = cache.pool.clone()
        gb.cache4_append(cache, K, V, slots)
        check(cache, before, K, V, slots)


@pytest.mark.parametrize("d", [64, 128])
def test_the_sign_of_a_zero_code(d):
    # to the bit, which a comparison of numbers does not see: that of the number, of zeros themselves too; none under a scale of zero
    g = torch.Generator().manual_seed(5)
    x = torch.randn(70, 2, d, generator=g) * torch.exp2(torch.randint(-30, 1, (70, 2, d), generator=g).float())
    x[::3] = torch.where(torch.rand(x[::3].shape, generator=g) < 0.5, -0.0, x[::3])
    x[5] = -1e-9
    K = x.bfloat16().cuda()
    cache = filled(2, 2, d, "e2m1")
    slots = torch.arange(70, device="cuda") + 3
    gb.cache4_append(cache, K, -K, slots)
    k, v, ks, vs = codes_and_scales(cache.pool, slots, "e2m1")
    assert int(((k == 0) & torch.signbit(k)).sum()) > 100
    for code, scale, want in ((k, ks, K), (v, vs, -K)):
        live = (scale > 0).repeat_interleave(GROUP, -1)
        assert torch.equal(torch.signbit(code), torch.signbit(want) & live)


@pytest.mark.parametrize("d", [64, 128])
def test_the_sign_of_what_becomes_zero(d):
    # e2m1 has a zero of either sign: that of the number, however small it is beside the group's largest
    small = [0.0, 2.0 ** -130, 2.0 ** -40, 2.0 ** -18, 2.0 ** -17, 2.0 ** -16, 2.0 ** -15, 2.0 ** -8, 0.125, 0.2421875, 0.25, 0.2578125]
    g = torch.Generator().manual_seed(4)
    x = torch.tensor(small)[torch.randint(len(small), (40, d), generator=g)] * torch.where(torch.rand(40, d, generator=g) < 0.5, -1.0, 1.0)
    x[:, 7::16] = torch.where(torch.rand(40, d // 16, generator=g) < 0.5, -6.0, 6.0)
    K = x[:, None].bfloat16().cuda()
    V = -K.flip(0).contiguous()
    slots = torch.arange(40, device="cuda")
    cache = filled(1, 1, d, "e2m1")
    before = cache.pool.clone()
    gb.cache4_append(cache, K, V, slots)
    check(cache, before, K, V, slots)
    k, v, _, _ = (t.cuda() for t in places(d, "e2m1"))
    flat = cache.pool.reshape(-1).int()
    for x, where in ((K, k), (V, v)):
        codes = flat[where[:40, :, 0]] >> where[:40, :, 1].int() & 15
        assert torch.equal(codes >= 8, torch.signbit(x[:, 0]))


@pytest.mark.parametrize("kind", KINDS)
def test_every_bf16_number_of_a_range(kind):
    # all 2^15 bf16 magnitudes from 2^-14 up to 2^7, in groups beside a fixed largest number
    d = 64
    x = torch.arange(0x3880, 0x4300, dtype=torch.int32)
    x = (x.to(torch.int16)).view(torch.bfloat16).float()
    n = -(-len(x) // (d // 2))
    x = torch.cat((x, torch.zeros(n * (d // 2) - len(x)))).view(n, d // 2)
    K = torch.zeros(n, d)
    K[:, 0::2], K[:, 1::2] = x, -x.flip(1)
    K[:, 15::16] = 90.0
    K = K[:, None].bfloat16().cuda()
    slots = torch.arange(n, device="cuda")
    cache = filled(-(-n // PAGE), 1, d, kind)
    before = cache.pool.clone()
    gb.cache4_append(cache, K, -K, slots)
    check(cache, before, K, -K, slots)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_group_that_cannot_be_held_is_nan(bad, kind):
    cache = filled(1, 2, 64, kind)
    before = cache.pool.clone()
    K, V = randn(3, 4, 2, 64), randn(4, 4, 2, 64)
    K[1, 0, 17] = V[2, 1, 63] = bad
    slots = slots_of(8, 9, 10, 11)
    gb.cache4_append(cache, K, V, slots)
    check(cache, before, K, V, slots)
    k, v = gb.cache4_read(cache, slots)
    assert bool(k[1, 0, 16:32].isnan().all()) and int(k.isnan().sum()) == 16
    assert bool(v[2, 1, 48:].isnan().all()) and int(v.isnan().sum()) == 16


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_append_does_not_depend_on_the_split(d, kind):
    H, N = 3, 333
    K, V = randn(5, N, H, d), randn(6, N, H, d)
    slots = torch.randperm(6 * PAGE, generator=torch.Generator().manual_seed(7))[:N].sort().values.cuda()
    once, pieces, single = (filled(6, H, d, kind, k_exp=-3) for _ in range(3))
    gb.cache4_append(once, K, V, slots)
    at = 0
    for n in (1, 30, 2, 64, 33, 100, 103):
        gb.cache4_append(pieces, K[at:at + n], V[at:at + n], slots[at:at + n])
        at += n
    for i in range(N):
        gb.cache4_append(single, K[i:i + 1], V[i:i + 1], slots[i:i + 1])
    assert torch.equal(once.pool, pieces.pool) and torch.equal(once.pool, single.pool)


def test_packed_rows_and_views():
    # keys and values as column blocks of one projection's output, and rows far apart
    H, d, N = 2, 128, 70
    packed = randn(8, N, 8 * d)
    K, V = packed[:, 4 * d:6 * d].unflatten(-1, (H, d)), packed[:, 6 * d:].unflatten(-1, (H, d))
    slots = torch.arange(10, 10 + N, device="cuda")
    a, b = filled(2, H, d, "e2m1"), filled(2, H, d, "e2m1")
    gb.cache4_append(a, K, V, slots)
    gb.cache4_append(b, K.contiguous(), V.contiguous(), slots)
    assert torch.equal(a.pool, b.pool)
    want = gb.cache4_read(a, slots)
    wide = torch.full((N, 8 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    out_k, out_v = wide[:, :2 * d].unflatten(-1, (H, d)), wide[:, 4 * d:6 * d].unflatten(-1, (H, d))
    gb.cache4_read(a, slots, out_k=out_k, out_v=out_v)
    assert torch.equal(out_k, want[0]) and torch.equal(out_v, want[1])
    assert bool((wide[:, 2 * d:4 * d] == 3).all()) and bool((wide[:, 6 * d:] == 3).all())
    for bad in (K[:, :1], K.transpose(1, 2), K[::2], K.float()):
        with pytest.raises(ValueError):
            gb.cache4_append(a, bad, V, slots)
    with pytest.raises(ValueError):
        gb.cache4_append(a, K, V, slots.int())
    with pytest.raises(ValueError):
        gb.cache4_append(a, K, V, slots[:-1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_read_gives_every_code_and_scale_back(d, kind):
    # random bytes: every code under every scale, NaN and negative scales among them
    H = 3
    cache = filled(3, H, d, kind, k_exp=-6, v_exp=5)
    cache.pool.copy_(torch.randint(0, 256, cache.pool.shape, generator=torch.Generator().manual_seed(9)).to(torch.uint8))
    slots = torch.cat((torch.randperm(3 * PAGE, generator=torch.Generator().manual_seed(10)).cuda(), slots_of(-1, 5, 5, -2, 191)))
    k, v = gb.cache4_read(cache, slots)
    at = slots.clamp(min=0)
    for got, want in zip((k, v), held(cache, at)):
        want = torch.where((slots >= 0)[:, None, None], want, 0.0)
        assert torch.equal(got.double().nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))


def test_read_undoes_the_append_of_what_can_be_held():
    # numbers that are codes times a scale: nothing is lost
    for kind in KINDS:
        table = torch.tensor(CODES[kind], dtype=torch.float32)
        g = torch.Generator().manual_seed(11)
        pick = torch.randint(1 if kind == "int4" else 0, 16, (50, 2, 128), generator=g)
        x = table[pick].unflatten(-1, (-1, GROUP))
        x[..., 0] = TOP[kind]
        x = (x * 2.0 ** torch.randint(-4, 5, x.shape[:-1], generator=g)[..., None]).flatten(-2).bfloat16().cuda()
        cache = filled(1, 2, 128, kind)
        slots = torch.arange(50, device="cuda")
        gb.cache4_append(cache, x, -x, slots)
        k, v = gb.cache4_read(cache, slots)
        assert torch.equal(k, x) and torch.equal(v, -x)


@pytest.mark.parametrize("what", ["append", "read"])
def test_slots_past_the_pool_are_passed_over(what):
    cache = filled(2, 2, 64, "e2m1", byte=0x22)
    slots = slots_of(3, 128, 2 ** 40, 5, -1)
    K, V = randn(12, 5, 2, 64), randn(13, 5, 2, 64)
    before = cache.pool.clone()
    if what == "append":
        gb.cache4_append(cache, K, V, slots)
        assert gb.check_device_error() == gb.ERR_CACHE_RANGE
        check(cache, before, K, V, slots_of(3, -1, -1, 5, -1))
    else:
        k, v = gb.cache4_read(cache, slots)
        assert gb.check_device_error() == gb.ERR_CACHE_RANGE
        assert not bool(k[[1, 2, 4]].any()) and not bool(v[[1, 2, 4]].any()) and bool(k[[0, 3]].any())


def test_no_rows():
    cache = filled(1, 1, 64, "int4")
    before = cache.pool.clone()
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    gb.cache4_append(cache, none, none, slots_of())
    k, v = gb.cache4_read(cache, slots_of())
    assert k.shape == v.shape == (0, 1, 64) and torch.equal(cache.pool, before)


def test_a_pool_of_more_than_32_bits_of_bytes():
    H, d = 8, 128
    n_pages = 2 ** 32 // (H * 72 * d) + 600
    cache = gb.cache4_alloc(n_pages, H, d, "e2m1", k_exp=-4)
    assert cache.pool.numel() > 2 ** 32
    slots = torch.cat([torch.arange(s, s + 40, device="cuda") for s in (0, 64 * (n_pages - 1) + 24, 64 * (n_pages - 300) + 5)])
    K, V = randn(14, 120, H, d), randn(15, 120, H, d)
    gb.cache4_append(cache, K, V, slots)
    small = filled(3, H, d, "e2m1", k_exp=-4)
    there = torch.cat([torch.arange(s, s + 40, device="cuda") for s in (0, 64 + 24, 128 + 5)])
    gb.cache4_append(small, K, V, there)
    for a, b in zip(gb.cache4_read(cache, slots), gb.cache4_read(small, there)):
        assert torch.equal(a, b)
    del cache
    torch.cuda.empty_cache()
