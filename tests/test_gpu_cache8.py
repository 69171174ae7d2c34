"""The 8-bit K/V cache: what the append writes, exactly, and the gated attention
over it against the 64-bit formula on the cache's own bytes.

Tolerances of the attention. A score is a sum of d_k exact products (8-bit codes
times at most 8 significant bits) in float32, whose order and truncation are the
tensor core's: off by at most d_k 2^-23 sum |q_c k_c| / sqrt(d_k), the same
share of the weight. A weight is rounded to fp16 (2^-11 of itself), in the open
block to bf16 (2^-8), before it multiplies V. Both errors weigh like the weights
themselves: with A = sum_j w_j |v_j| the output is off by at most
(half step + 2 score error) A, twice the score's because the denominator has it
too; exponentials and the gate's sigmoid add 2^-20; the store rounds to bf16.
"""
import math

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from ops_ref import BLOCK, RefCache, attend, cache_rows, code_values, frequencies, half_step, norm_rope, quantise

pytestmark = pytest.mark.gpu
KINDS = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    gb.load()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert gb.check_device_error() == gb.OK


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(B, capacity, H, d, kind):
    """A cache whose every byte is something that must not be used."""
    c = gb.cache8_alloc(B, capacity, H, d, kind)
    for t in (c.k8, c.v8):
        t.view(torch.uint8).fill_(0x7F)              # e4m3: NaN
    for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail):
        t.fill_(float("nan"))
    return c


def bytes_of(c):
    return [t.view(torch.uint8).clone() for t in (c.k8, c.v8, c.k_scale, c.v_scale, c.k_tail, c.v_tail)]


def rows(B, L, H, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(B, L, H, d, generator=g)).bfloat16().cuda()


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=12345.0), torch.nan_to_num(b.double(), nan=12345.0))


def check_block(cache, b, h, j, k, v):
    """Block j of (b, h) holds exactly the codes and scales of its 64 rows."""
    for codes, scale, x, turn in ((cache.k8, cache.k_scale, k, False), (cache.v8, cache.v_scale, v, True)):
        q, s = quantise(x.double().cpu(), "int8" if codes.dtype == torch.int8 else "e4m3")
        got = code_values(codes[b, h, j])
        assert torch.equal(got.T if turn else got, q), (b, h, j, turn)
        assert same(scale[b, h, j].cpu().reshape(1), torch.tensor([s], dtype=torch.float32)), (b, h, j, turn)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,d", [(1, 64), (3, 128)])
def test_append_in_pieces_holds_exactly_the_formula(kind, H, d):
    # four sequences, steps of uneven length: single tokens, none, pieces that close no, one
    # and several blocks, that end with a block, and that start inside one
    B, capacity = 4, 448
    steps = [(3, [3, 0, 1, 2]), (70, [70, 64, 5, 63]), (1, [1, 0, 1, 1]), (130, [130, 128, 127, 1]), (64, [60, 64, 1, 63]),
             (66, [65, 0, 66, 2])]
    cache = filled(B, capacity, H, d, kind)
    all_k = [torch.zeros(0, H, d).bfloat16().cuda() for _ in range(B)]
    all_v = [torch.zeros(0, H, d).bfloat16().cuda() for _ in range(B)]
    lens = [0] * B
    for n, (L, new) in enumerate(steps):
        K, V = rows(B, L, H, d, 10 + n, 0.3 + n), rows(B, L, H, d, 50 + n, 2.0 ** (n - 3))
        before = bytes_of(cache)
        gb.cache8_append(cache, K, V, ints(*lens), ints(*new))
        after = bytes_of(cache)
        for b in range(B):
            all_k[b], all_v[b] = torch.cat((all_k[b], K[b, :new[b]])), torch.cat((all_v[b], V[b, :new[b]]))
            old, end = lens[b], lens[b] + new[b]
            for h in range(H):
                for j in range(capacity // BLOCK):
                    if old // BLOCK <= j < end // BLOCK:
                        check_block(cache, b, h, j, all_k[b][j * BLOCK:(j + 1) * BLOCK, h],
                                    all_v[b][j * BLOCK:(j + 1) * BLOCK, h])
                    else:   # every other block as it was
                        assert all(torch.equal(before[i][b, h, j], after[i][b, h, j]) for i in (0, 1)), (b, h, j)
                        assert all(torch.equal(before[i].view(B, H, -1, 4)[b, h, j], after[i].view(B, H, -1, 4)[b, h, j])
                                   for i in (2, 3))
                # the last two touched blocks' new tokens are in the open-block buffers, the rest as it was
                want_k, want_v = before[4].view(torch.bfloat16)[b, h].clone(), before[5].view(torch.bfloat16)[b, h].clone()
                last = (end - 1) // BLOCK
                for p in range(max(old, (last - 1) * BLOCK), end):
                    want_k[p // BLOCK % 2, p % BLOCK] = all_k[b][p, h]
                    want_v[p // BLOCK % 2, :, p % BLOCK] = all_v[b][p, h]
                assert same(cache.k_tail[b, h], want_k) and same(cache.v_tail[b, h], want_v), (b, h)
            lens[b] = end


@pytest.mark.parametrize("kind", KINDS)
def test_append_does_not_depend_on_the_split(kind):
    B, H, d, L = 2, 2, 128, 200
    K, V = rows(B, L, H, d, 1), rows(B, L, H, d, 2)
    once, steps = filled(B, 256, H, d, kind), filled(B, 256, H, d, kind)
    gb.cache8_append(once, K, V, ints(0, 0))
    for i in range(L):
        gb.cache8_append(steps, K[:, i:i + 1], V[:, i:i + 1], ints(i, i))
    full, rest = L // BLOCK, L % BLOCK
    for a, b in ((once, steps),):
        assert torch.equal(a.k8[:, :, :full].view(torch.uint8), b.k8[:, :, :full].view(torch.uint8))
        assert torch.equal(a.v8[:, :, :full].view(torch.uint8), b.v8[:, :, :full].view(torch.uint8))
        assert torch.equal(a.k_scale[:, :, :full], b.k_scale[:, :, :full])
        assert torch.equal(a.k_tail[:, :, full % 2, :rest], b.k_tail[:, :, full % 2, :rest])
        assert torch.equal(a.v_tail[:, :, full % 2, :, :rest], b.v_tail[:, :, full % 2, :, :rest])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_append_of_long_prompts_is_that_of_short_pieces(kind, d):
    # more blocks than the GPU holds at once, from inside a block on; against pieces of at most 64 tokens
    B, H, capacity, start = 5, 8, 1280, [0, 63, 64, 17, 100]
    new = [1100, 1025, 1, 1047, 1100]
    K, V = rows(B, 1200, H, d, 21), rows(B, 1200, H, d, 22, 3.0)
    one, many = filled(B, capacity, H, d, kind), filled(B, capacity, H, d, kind)
    for c in (one, many):
        gb.cache8_append(c, K[:, :100].contiguous(), V[:, :100].contiguous(), ints(*[0] * B), ints(*start))
    late_k, late_v = K[:, 100:].contiguous(), V[:, 100:].contiguous()
    gb.cache8_append(one, late_k, late_v, ints(*start), ints(*new))
    for at in range(0, 1100, 64):
        n = [max(0, min(64, x - at)) for x in new]
        gb.cache8_append(many, late_k[:, at:at + 64].contiguous(), late_v[:, at:at + 64].contiguous(),
                         ints(*[s + min(at, x) for s, x in zip(start, new)]), ints(*n))
    for b in range(B):
        for h in range(H):
            for x, y in zip(cache_rows(one, b, h, start[b] + new[b]), cache_rows(many, b, h, start[b] + new[b])):
                assert torch.equal(x, y), (b, h)


@pytest.mark.parametrize("kind", KINDS)
def test_append_takes_back_up_to_64_tokens(kind):
    H, d = 2, 64
    K, V = rows(1, 300, H, d, 3), rows(1, 300, H, d, 4)
    K2, V2 = rows(1, 90, H, d, 5), rows(1, 90, H, d, 6)
    for end in (128, 129, 160, 191, 192, 193):
        for back in (1, 17, 63, 64):
            cache, want = filled(1, 320, H, d, kind), filled(1, 320, H, d, kind)
            gb.cache8_append(cache, K[:, :end - 30], V[:, :end - 30], ints(0))
            gb.cache8_append(cache, K[:, end - 30:end], V[:, end - 30:end], ints(end - 30))
            T = end - back
            gb.cache8_append(cache, K2, V2, ints(T))
            gb.cache8_append(want, torch.cat((K[:, :T], K2), 1), torch.cat((V[:, :T], V2), 1), ints(0))
            for h in range(H):
                for x, y in zip(cache_rows(cache, 0, h, T + 90), cache_rows(want, 0, h, T + 90)):
                    assert torch.equal(x, y), (end, back)


@pytest.mark.parametrize("kind", KINDS)
def test_append_edge_values(kind):
    # one block per case, in K and, shifted by one case, in V
    d = 64
    g = torch.Generator().manual_seed(7)
    base = torch.randn(BLOCK, d, generator=g)
    ties = (torch.arange(BLOCK * d).view(BLOCK, d) % 254 - 126.5).bfloat16().float()   # with 127: scale 1, halves
    ties[0, 0] = 127.0
    borders = torch.linspace(-448, 448, BLOCK * d).view(BLOCK, d)                       # many e4m3 midpoints
    cases = [torch.zeros(BLOCK, d), base * 1e-38, base * 3e-40, base * 1e37, base.clamp(-3, 3) * 1.1e38, ties, borders,
             borders * 2.0 ** -9, torch.where(base > 3.0, base * 1e30, base * 1e-3), base.clone(), base.clone(),
             torch.full((BLOCK, d), 2.0 ** -133)]
    cases[9][5, 6], cases[10][63, 63] = float("nan"), float("-inf")
    x = torch.stack(cases).bfloat16().cuda()                            # [n, 64, d]
    n = len(cases)
    K = x.reshape(1, n * BLOCK, 1, d)
    V = torch.roll(x, 1, 0).reshape(1, n * BLOCK, 1, d)
    cache = filled(1, n * BLOCK, 1, d, kind)
    gb.cache8_append(cache, K, V, ints(0))
    for j in range(n):
        check_block(cache, 0, 0, j, x[j], x[j - 1])


def test_append_of_column_blocks_of_a_projection():
    B, L, H, d = 2, 70, 4, 128
    g = torch.Generator().manual_seed(8)
    packed = torch.randn(B, L, 6 * H * d, generator=g).bfloat16().cuda()
    K = packed[..., 4 * H * d:5 * H * d].unflatten(-1, (H, d))
    V = packed[..., 5 * H * d:].unflatten(-1, (H, d))
    a, b = gb.cache8_alloc(B, 128, H, d), gb.cache8_alloc(B, 128, H, d)
    gb.cache8_append(a, K, V, ints(0, 0), ints(70, 64))
    gb.cache8_append(b, K.contiguous(), V.contiguous(), ints(0, 0), ints(70, 64))
    for h in range(H):
        for s, T in ((0, 70), (1, 64)):
            assert all(torch.equal(x, y) for x, y in zip(cache_rows(a, s, h, T), cache_rows(b, s, h, T)))


def test_append_leaves_sequences_that_do_not_fit():
    B, H, d = 6, 1, 64
    K, V = rows(B, 70, H, d, 9), rows(B, 70, H, d, 10)
    cache = filled(B, 128, H, d, "int8")
    before = bytes_of(cache)
    lens, new = ints(-1, 59, 128, 2 ** 31 - 1, 58, 0), ints(5, 70, 1, 70, 70, 71)
    gb.cache8_append(cache, K, V, lens, new)
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert gb.check_device_error() == gb.OK                 # read and cleared
    after = bytes_of(cache)
    for i, (x, y) in enumerate(zip(before, after)):
        x, y = x.reshape(B, -1), y.reshape(B, -1)
        assert all(torch.equal(x[b], y[b]) for b in (0, 1, 2, 3, 5)), i
    check = gb.cache8_alloc(1, 128, H, d)                   # the one that fits has its rows
    assert not torch.equal(before[0][4], after[0][4])
    del check
    gb.cache8_append(cache, K, V, ints(*[0] * 6), ints(*[-1] * 6))
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE


# ---------------------------------------------------------------- attention
def gate_inputs(gate, B, Lq, Hq, d, dm, seed):
    if gate == "none":
        return None, None
    g = torch.Generator().manual_seed(seed)
    cols = Hq if gate == "headwise" else Hq * d
    return (torch.randn(B, Lq, dm, generator=g).bfloat16().cuda(),
            (torch.randn(dm, cols, generator=g) / math.sqrt(dm)).bfloat16().cuda())


def fill_cache(lens_after, H, d, kind, seed, capacity=None, scale=1.0):
    """A cache of sequences of these lengths, through the append."""
    B, L = len(lens_after), max(max(lens_after), 1)
    capacity = capacity or (L + BLOCK - 1) // BLOCK * BLOCK
    cache = filled(B, capacity, H, d, kind)
    gb.cache8_append(cache, rows(B, L, H, d, seed, scale), rows(B, L, H, d, seed + 1, scale), ints(*[0] * B),
                     ints(*lens_after))
    return cache


def check_attention(O, X, Q, cache, W_g, gate, lens, new):
    B, Lq, Hq, d = Q.shape
    H, G = cache.H_kv, Hq // cache.H_kv
    for b in range(B):
        T = lens[b] + new[b]
        assert not bool(O[b, new[b]:].any()), f"rows past n_new of sequence {b} are not zero"
        if new[b] == 0:
            continue
        sig = torch.ones(new[b], Hq, d, dtype=torch.float64)
        if gate != "none":
            s = torch.sigmoid(X[b, :new[b]].double() @ W_g.double()).cpu()
            sig = s[..., None].expand(-1, -1, d) if gate == "headwise" else s.view(new[b], Hq, d)
        for h in range(H):
            k, v = (t.cpu() for t in cache_rows(cache, b, h, T))
            q = Q[b, :new[b], h * G:(h + 1) * G].double().cpu().reshape(-1, d)
            seen = [lens[b] + r // G + 1 for r in range(new[b] * G)]
            ref, mag, top = attend(q, k, v, seen)
            got = O[b, :new[b], h * G:(h + 1) * G].double().cpu().reshape(-1, d)
            gt = sig[:, h * G:(h + 1) * G].reshape(-1, d)
            ref, mag = ref * gt, mag * gt
            weight = half_step(torch.bfloat16) if T % BLOCK else half_step(torch.float16)
            tol = half_step(torch.bfloat16) * ref.abs() + (weight + 2 * d * 2.0 ** -23 * top[:, None] + 2.0 ** -20) * mag
            err = (got - ref).abs()
            assert bool((err <= tol + 1e-30).all()), (b, h, T, float((err / (tol + 1e-30)).max()))


CASES = [
    # lens before, rows, new rows (None: all), Hq, Hkv, d, kind, gate
    ([0], 1, None, 1, 1, 64, "int8", "none"),
    ([0, 62, 63, 64, 127, 128, 200], 1, None, 4, 2, 128, "int8", "none"),
    ([0, 62, 63, 64, 127, 128, 200], 1, None, 8, 1, 64, "e4m3", "headwise"),
    ([1000], 1, None, 32, 8, 128, "int8", "elementwise"),
    ([5, 700, 64, 63], 1, [1, 1, 0, 1], 14, 2, 128, "e4m3", "elementwise"),
    ([60, 0, 1, 500], 5, None, 8, 2, 128, "int8", "none"),
    ([60, 0, 130, 500], 8, [8, 3, 0, 5], 8, 2, 64, "e4m3", "headwise"),
    ([63, 640], 16, [16, 1], 8, 1, 128, "int8", "none"),            # 128 rows: 8 warps to a tile
    ([100, 3], 70, [70, 66], 1, 1, 128, "e4m3", "none"),            # more rows than a block, 5 groups of 16
    ([30, 300, 3000], 3, None, 24, 2, 64, "int8", "elementwise"),   # 36 rows: 4 warps to a tile
    ([40, 1111], 2, None, 20, 2, 128, "int8", "none"),              # 20 rows: 2 warps to a tile
    ([33333], 1, None, 16, 2, 128, "e4m3", "none"),                 # one sequence split over every SM
    ([20001, 7, 0, 9999], 1, None, 4, 4, 64, "int8", "headwise"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][-1]}x{c[1]}-{c[3]}-{c[4]}-{c[5]}-{c[6]}-{c[7]}")
def test_attention(case):
    lens, Lq, new, Hq, H, d, kind, gate = case
    if gate == "headwise" and Hq % 8:
        Hq, H = 8 * H, H
    B = len(lens)
    n = new or [Lq] * B
    cache = fill_cache([a + b for a, b in zip(lens, n)], H, d, kind, 21)
    Q = rows(B, Lq, Hq, d, 23, 1.5)
    X, W = gate_inputs(gate, B, Lq, Hq, d, 256, 24)
    O = gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W, gate=gate, n_new=None if new is None else ints(*new))
    check_attention(O, X, Q, cache, W, gate, lens, n)


def test_attention_many_sequences_of_every_length():
    # more sequences than threads in a CTA, most short, some empty
    g = torch.Generator().manual_seed(30)
    B = 601
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    new = torch.randint(0, 3, (B,), generator=g).tolist()
    lens[17], lens[600] = 1500, 777
    new[600] = 2
    cache = fill_cache([a + b for a, b in zip(lens, new)], 1, 64, "int8", 31)
    Q = rows(B, 2, 2, 64, 32)
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(*lens), gate="none", n_new=ints(*new))
    check_attention(O, None, Q, cache, None, "none", lens, new)


@pytest.mark.parametrize("kind,Lq,G,gate", [("int8", 1, 4, "headwise"), ("e4m3", 1, 8, "none"), ("int8", 3, 4, "none")])
def test_attention_heads_cut_into_few_parts(kind, Lq, G, gate):
    # so many tiles that a team's share is of the order of a head: heads within a share, cut once,
    # and cut several times, which the teams merge themselves
    g = torch.Generator().manual_seed(35)
    B, H, d = 24, 8, 64
    lens = torch.randint(600, 2600, (B,), generator=g).tolist()
    lens[3], lens[4], lens[11] = 0, 63, 2559
    n = [Lq] * B
    n[7] = 0
    cache = fill_cache([a + b for a, b in zip(lens, n)], H, d, kind, 36)
    Q = rows(B, Lq, H * G, d, 37, 1.5)
    X, W = gate_inputs(gate, B, Lq, H * G, d, 256, 38)
    O = gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W, gate=gate, n_new=ints(*n))
    check_attention(O, X, Q, cache, W, gate, lens, n)
    assert torch.equal(O, gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W, gate=gate, n_new=ints(*n)))


@pytest.mark.parametrize("lens", [[1023, 0, 700], [1024], [1087, 3], [64 * 128]])
def test_attention_in_a_cache_much_longer_than_its_sequences(lens):
    # the grid is planned for the capacity; 16 tiles and 17 are on either side of a CTA to a head,
    # 128 of a merge in one and in two levels
    B, H, d = len(lens), 2, 128
    cache = fill_cache([n + 1 for n in lens], H, d, "int8", 45, capacity=64 * 1024)
    Q = rows(B, 1, 8, d, 46, 1.5)
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(*lens), gate="none")
    check_attention(O, None, Q, cache, None, "none", lens, [1] * B)


@pytest.mark.parametrize("kind,d,H,G,Lq,gate", [("e4m3", 128, 2, 8, 1, "headwise"), ("int8", 64, 3, 2, 2, "elementwise"),
                                               ("int8", 128, 1, 16, 3, "none"), ("e4m3", 64, 2, 32, 4, "none")])
def test_attention_heads_in_many_parts_beside_short_ones(kind, d, H, G, Lq, gate):
    # long heads cut into more parts than a thread merges at once, between heads of a few tiles, whose
    # ends (with and without an open block) and the places after them fall anywhere in the teams' shares
    lens_after = [40001, 5, 64, 129, 3 * 64, 0, 40000, 1, 700, 64 * 40]
    n = [min(Lq, x) for x in lens_after]
    cache = fill_cache(lens_after, H, d, kind, 91)
    X, W_g = gate_inputs(gate, len(n), Lq, H * G, d, 256, 92)
    Q = rows(len(n), Lq, H * G, d, 93)
    lens = [x - y for x, y in zip(lens_after, n)]
    O = gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W_g, gate=gate, n_new=ints(*n))
    check_attention(O, X, Q, cache, W_g, gate, lens, n)


@pytest.mark.parametrize("H,d,Lq,G,gate", [(8, 64, 1, 4, "none"), (2, 128, 2, 8, "headwise")])
def test_attention_more_heads_than_teams(H, d, Lq, G, gate):
    # thousands of short heads, most of them a team's alone, empty sequences between them; and one long enough
    # to be cut into several parts
    g = torch.Generator().manual_seed(94)
    lens_after = [int(x) for x in torch.randint(0, 400, (700,), generator=g)]
    for b in range(0, 700, 9):
        lens_after[b] = 0
    lens_after[333], lens_after[699] = 64 * 50 + 3, 64
    n = [min(Lq, x) for x in lens_after]
    B, capacity = 700, 64 * 51
    cache = filled(B, capacity, H, d, "int8")
    step = 448
    K, V = rows(B, step, H, d, 95), rows(B, step, H, d, 96)
    for at in range(0, capacity, step):
        gb.cache8_append(cache, K, V, ints(*[min(at, x) for x in lens_after]),
                         ints(*[max(0, min(step, x - at)) for x in lens_after]))
    X, W_g = gate_inputs(gate, B, Lq, H * G, d, 64, 97)
    Q = rows(B, Lq, H * G, d, 98)
    lens = [x - y for x, y in zip(lens_after, n)]
    O = gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W_g, gate=gate, n_new=ints(*n))
    for b in [0, 1, 9, 332, 333, 334, 500, 698, 699]:
        one = gb.Cache8(*(t[b:b + 1] for t in (cache.k8, cache.v8, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail)))
        x = None if X is None else X[b:b + 1]
        check_attention(O[b:b + 1], x, Q[b:b + 1], one, W_g, gate, [lens[b]], [n[b]])
    check = list(range(0, B, 7)) + [333]
    got = O[check].double()
    part = gb.Cache8(*(t[check].contiguous() for t in (cache.k8, cache.v8, cache.k_scale, cache.v_scale, cache.k_tail,
                                                        cache.v_tail)))
    again = gb.gated_sdpa_cache8(None if X is None else X[check].contiguous(), Q[check].contiguous(), part,
                                 ints(*[lens[b] for b in check]), W_g, gate=gate, n_new=ints(*[n[b] for b in check])).double()
    # the same sums cut elsewhere: each side within 2^-7 of the largest value of the definition (bf16's half step
    # 2^-9, the weights' 2^-9 for the open block, both of values no larger than that)
    assert float((got - again).abs().max()) <= 2.0 ** -6 * float(again.abs().max())


def test_attention_nothing_to_do_and_repeats():
    cache = fill_cache([5, 70], 2, 64, "int8", 33)
    Q = rows(2, 1, 4, 64, 34)
    out = torch.full_like(Q, float("nan"))
    gb.gated_sdpa_cache8(None, Q, cache, ints(5, 70), gate="none", n_new=ints(0, 0), out=out)
    assert not bool(out.any())
    cache = fill_cache([4097, 70], 2, 64, "int8", 33)
    a = gb.gated_sdpa_cache8(None, Q, cache, ints(4096, 69), gate="none")
    assert all(torch.equal(a, gb.gated_sdpa_cache8(None, Q, cache, ints(4096, 69), gate="none")) for _ in range(5))


def test_attention_value_scales_far_apart():
    # a block of values 2^40 times larger that the query gives weights of about e^-60, blocks of
    # zeros and of tiny values: each output stays as exact as its own weights
    H, d, T = 1, 128, 64 * 6 + 10
    K, V = rows(1, T, H, d, 40), rows(1, T, H, d, 41)
    Q = rows(1, 1, 4, d, 42)
    away = -Q[0, 0].double().mean(0)
    away = away / away.norm()
    K[0, 128:192, 0] += (200 * away).bfloat16()
    V[0, 128:192] *= 2.0 ** 40
    V[0, 192:256] = 0
    V[0, 256:320] *= 2.0 ** -100
    cache = filled(1, 512, H, d, "e4m3")
    gb.cache8_append(cache, K, V, ints(0))
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(T - 1), gate="none")
    check_attention(O, None, Q, cache, None, "none", [T - 1], [1])
    # nothing but zeros to see
    V.zero_()
    gb.cache8_append(cache, K, V, ints(0))
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(T - 1), gate="none")
    assert not bool(O.any())


def test_attention_large_and_tiny_queries():
    H, d, T = 2, 64, 333
    cache = fill_cache([T], H, d, "int8", 43)
    Q = rows(1, 1, 8, d, 44)
    Q[0, 0, 1] *= 64           # one token takes nearly all the weight
    Q[0, 0, 2] *= 2.0 ** -120  # even weights
    Q[0, 0, 3] = 0
    Q[0, 0, 4, :32] *= 2.0 ** -20
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(T - 1), gate="none")
    check_attention(O, None, Q, cache, None, "none", [T - 1], [1])


@pytest.mark.parametrize("kind", KINDS)
def test_attention_non_finite_blocks_reach_only_the_rows_that_see_them(kind):
    H, d, Lq, T = 1, 64, 6, 131
    lens = T - Lq                                            # 125: rows 0..2 end with block 1, rows 3.. see block 2
    K, V = rows(2, T, H, d, 50), rows(2, T, H, d, 51)
    V[0, 127, 0, 9] = float("inf")                           # the token that row 2 adds: spoils block 1 for all
    K2, V2 = K.clone(), V.clone()
    cache = filled(2, 192, H, d, kind)
    gb.cache8_append(cache, K2, V2, ints(0, 0))
    Q = rows(2, Lq, 4, d, 52)
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(lens, lens), gate="none")
    assert bool(torch.isnan(O[0]).all())
    check_attention(O[1:], None, Q[1:], Cache8View(cache, 1), None, "none", [lens], [Lq])
    # a NaN in block 2, closed by the step itself: rows before it keep their values
    L2 = 70                                                  # tokens 122 .. 191: rows 0..5 see blocks 0, 1 only
    K, V = rows(1, 192, H, d, 53), rows(1, 192, H, d, 54)
    K[0, 150, 0, 3] = float("nan")
    V[0, 180, 0, 3] = float("nan")
    cache = filled(1, 192, H, d, kind)
    gb.cache8_append(cache, K, V, ints(0))
    Q = rows(1, L2, 1, d, 55)
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(192 - L2), gate="none")
    first = 128 - (192 - L2)                                 # first row that sees block 2
    assert bool(torch.isnan(O[0, first:]).all()) and not bool(torch.isnan(O[0, :first]).any())
    n = torch.tensor([first], dtype=torch.int32, device="cuda")
    again = gb.gated_sdpa_cache8(None, Q, cache, ints(192 - L2), gate="none", n_new=n)
    check_attention(again, None, Q, cache, None, "none", [192 - L2], [first])
    # (bits may differ: the tiles are dealt out differently)
    assert float((O[0, :first].double() - again[0, :first].double()).abs().max()) <= 0.02


class Cache8View:
    """One sequence of a cache, for the checks."""

    def __init__(self, c, b):
        for n in ("k8", "v8", "k_scale", "v_scale", "k_tail", "v_tail"):
            setattr(self, n, getattr(c, n)[b:b + 1])
        self.H_kv, self.d_k = c.H_kv, c.d_k


def test_attention_sequences_that_do_not_fit_are_zero():
    cache = fill_cache([100, 100, 100, 100], 1, 64, "int8", 60, capacity=128)
    Q = rows(4, 2, 2, 64, 61)
    lens, new = [-5, 127, 98, 2 ** 31 - 1], [2, 2, 2, 2]
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(*lens), gate="none", n_new=ints(*new))
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert not bool(O[0].any()) and not bool(O[1].any()) and not bool(O[3].any())
    check_attention(O[2:3], None, Q[2:3], Cache8View(cache, 2), None, "none", [98], [2])


def test_captured_steps_replay_with_new_lengths():
    # one graph of append + attention, replayed token by token; lens is moved in the graph too
    B, H, G, d, dm = 3, 2, 4, 128, 128
    cache = filled(B, 192, H, d, "int8")
    first = [0, 60, 125]
    g = torch.Generator().manual_seed(70)
    allK, allV = rows(B, 192, H, d, 71), rows(B, 192, H, d, 72)
    gb.cache8_append(cache, allK, allV, ints(0, 0, 0), ints(*first))
    lens = ints(*first)
    K, V, Q = (torch.zeros(B, 1, n, d, device="cuda", dtype=torch.bfloat16) for n in (H, H, G * H))
    X, W = gate_inputs("headwise", B, 1, G * H, d, dm, 73)
    ws = torch.empty(gb.cache8_workspace_bytes(cache, 1, G * H, dm, "headwise"), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(Q)
    gb.gated_sdpa_cache8(X, Q, cache, lens, W, gate="headwise", n_new=ints(0, 0, 0), out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gb.cache8_append(cache, K, V, lens)
        gb.gated_sdpa_cache8(X, Q, cache, lens, W, gate="headwise", out=out, workspace=ws)
        lens.add_(1)
    at = list(first)
    for step in range(8):
        for b in range(B):
            K[b, 0], V[b, 0] = allK[b, at[b]], allV[b, at[b]]
        Q.copy_(torch.randn(Q.shape, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, X, Q, cache, W, "headwise", at, [1] * B)
        at = [x + 1 for x in at]


def test_two_streams_with_workspaces_of_their_own():
    caches = [fill_cache([3000 + i, 10], 2, 64, "int8", 80 + i) for i in range(2)]
    Qs = [rows(2, 1, 8, 64, 82 + i) for i in range(2)]
    lens = [ints(2999 + i, 9) for i in range(2)]
    want = [gb.gated_sdpa_cache8(None, Qs[i], caches[i], lens[i], gate="none") for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(gb.cache8_workspace_bytes(caches[i], 1, 8, 0, "none"), dtype=torch.uint8, device="cuda")
          for i in range(2)]
    outs = [[torch.empty_like(Qs[i]) for _ in range(10)] for i in range(2)]
    for n in range(10):
        for i in range(2):
            gb.gated_sdpa_cache8(None, Qs[i], caches[i], lens[i], gate="none", out=outs[i][n], workspace=ws[i],
                                 stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i][n], want[i]) for i in range(2) for n in range(10))


def test_kept_workspaces_beside_a_graph_and_on_another_stream():
    # eager calls keep a workspace for each stream, a captured call has its own: replays in between
    # calls, and calls on a second stream at the same time, do not disturb them
    cache = fill_cache([5000, 200], 2, 128, "e4m3", 85)
    Q = rows(2, 1, 8, 128, 86)
    lens = ints(4999, 199)
    want = gb.gated_sdpa_cache8(None, Q, cache, lens, gate="none")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        captured = gb.gated_sdpa_cache8(None, Q, cache, lens, gate="none")
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        with torch.cuda.stream(side):
            graph.replay()
        outs.append(gb.gated_sdpa_cache8(None, Q, cache, lens, gate="none"))
        outs.append(gb.gated_sdpa_cache8(None, Q, cache, lens, gate="none", stream=side))
    torch.cuda.synchronize()
    assert torch.equal(captured, want) and all(torch.equal(o, want) for o in outs)


def test_append_fewer_tokens_than_rows_of_a_padded_batch():
    # L rows of K and V, more than the cache has room for; n_new of them are tokens
    H, d = 2, 128
    K, V = rows(3, 300, H, d, 12), rows(3, 300, H, d, 13)
    cache = filled(3, 128, H, d, "int8")
    gb.cache8_append(cache, K, V, ints(0, 0, 0), ints(128, 65, 0))
    gb.cache8_append(cache, K[:, 200:].contiguous(), V[:, 200:].contiguous(), ints(128, 65, 0), ints(0, 63, 1))
    want = filled(3, 128, H, d, "int8")
    for b, parts in enumerate([[(0, 128)], [(0, 65), (200, 263)], [(200, 201)]]):
        k, v = (torch.cat([t[b:b + 1, i:j] for i, j in parts], 1) for t in (K, V))
        T = k.shape[1]
        gb.cache8_append(want, k.expand(3, -1, -1, -1).contiguous(), v.expand(3, -1, -1, -1).contiguous(), ints(0, 0, 0),
                         ints(*[T if x == b else 0 for x in range(3)]))
        for h in range(H):
            assert all(torch.equal(x, y) for x, y in zip(cache_rows(cache, b, h, T), cache_rows(want, b, h, T)))


def test_refusals():
    cache = gb.cache8_alloc(2, 128, 2, 64)
    Q = torch.zeros(2, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    K = torch.zeros(2, 3, 2, 64, device="cuda", dtype=torch.bfloat16)
    lens = ints(0, 0)
    with pytest.raises(ValueError):
        gb.cache8_append(cache, K, K[:, :2], lens)
    with pytest.raises(ValueError):
        gb.cache8_append(cache, K[..., :1, :], K[..., :1, :], lens)
    with pytest.raises(ValueError):
        gb.cache8_append(cache, K.float(), K.float(), lens)
    with pytest.raises(ValueError):
        gb.cache8_append(cache, K, K, lens.long())
    with pytest.raises(ValueError):
        gb.cache8_append(cache, K, K, None)
    with pytest.raises(ValueError):
        gb.gated_sdpa_cache8(None, Q[:1], cache, lens, gate="none")
    with pytest.raises(ValueError):
        gb.gated_sdpa_cache8(None, Q, cache, lens[:1], gate="none")
    with pytest.raises(ValueError):
        gb.gated_sdpa_cache8(None, Q, cache, lens, gate="headwise")                       # no X
    for bad, st in ((Q.expand(2, 1, 4, 64).repeat(1, 65, 1, 1), gb.ERR_UNSUPPORTED),       # 130 query rows per head
                    (torch.zeros(2, 1, 3, 64, device="cuda", dtype=torch.bfloat16), gb.ERR_INVALID_ARG)):
        with pytest.raises(gb.GsdpaError) as e:
            gb.gated_sdpa_cache8(None, bad, cache, lens, gate="none")
        assert e.value.status == st
    with pytest.raises(gb.GsdpaError) as e:
        gb.gated_sdpa_cache8(None, Q, cache, lens, gate="none", workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gb.ERR_WORKSPACE
    wide = gb.cache8_alloc(2, 128, 2, 128)
    with pytest.raises(ValueError):   # v8 not transposed (with d_k = 64 the two shapes are one)
        gb.Cache8(wide.k8, wide.k8, wide.k_scale, wide.v_scale, wide.k_tail, wide.v_tail)
    with pytest.raises(ValueError):
        gb.Cache8(cache.k8, cache.v8, cache.k_scale, cache.v_scale[:, :, :1], cache.k_tail, cache.v_tail)


def test_waits_that_run_out_are_reported_and_leave_nothing_behind():
    # with a limit of 1 ns any wait that is not over within its first tries gives up: the calls report
    # OK or a timeout, never a fault, and the next ones with the default limit are right
    cache = fill_cache([30000, 700, 64 * 16], 2, 128, "int8", 87)
    Q = rows(3, 1, 8, 128, 88)
    lens, n = [29999, 699, 64 * 16 - 1], [1, 1, 1]
    G = 2000
    x, dx = rows(1, G, 6, 128, 89), rows(1, G, 6, 128, 90)
    rope = gb.Rope(128)
    want = gb.qk_norm_rope_bwd(x, x[:, :, :2].contiguous(), dx, dx[:, :, :2].contiguous(), rope=rope)
    statuses = []
    for _ in range(3):
        gb.set_wait_limit_ns(1)
        try:
            gb.gated_sdpa_cache8(None, Q, cache, ints(*lens), gate="none")
            statuses.append(gb.check_device_error())
            gb.qk_norm_rope_bwd(x, x[:, :, :2].contiguous(), dx, dx[:, :, :2].contiguous(), rope=rope)
            statuses.append(gb.check_device_error())
        finally:
            gb.set_wait_limit_ns(0)
        O = gb.gated_sdpa_cache8(None, Q, cache, ints(*lens), gate="none")
        got = gb.qk_norm_rope_bwd(x, x[:, :, :2].contiguous(), dx, dx[:, :, :2].contiguous(), rope=rope)
        assert gb.check_device_error() == gb.OK
        check_attention(O, None, Q, cache, None, "none", lens, n)
        assert all(torch.equal(got[k], want[k]) for k in want)
    assert set(statuses) <= {gb.OK, gb.ERR_DEVICE_TIMEOUT}


# ---------------------------------------------------------------- together, as they are used
@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_and_decoding_steps_together(kind):
    # projection rows -> norm and rotary positions -> cache -> gated attention, for a
    # prompt and steps of one and of three (drafted) tokens; the reference follows in 64 bits from
    # the bf16 values that the norm returned (its own error has tests of its own)
    B, H, G, d, dm = 2, 2, 4, 128, 256
    Hq = H * G
    rope, w = gb.Rope(64, layout="half"), frequencies(64)
    gam = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(90))).bfloat16().cuda()
    cache = filled(B, 256, H, d, kind)
    held = [[RefCache(kind, d) for _ in range(H)] for _ in range(B)]
    lens = [0, 0]
    for step, (L, new) in enumerate([(90, [90, 61]), (1, [1, 1]), (1, [1, 1]), (3, [3, 2]), (1, [1, 1]), (3, [1, 3])]):
        g = torch.Generator().manual_seed(91 + step)
        packed = torch.randn(B, L, (Hq + 2 * H) * d, generator=g).bfloat16().cuda()
        Q = packed[..., :Hq * d].unflatten(-1, (Hq, d))
        K = packed[..., Hq * d:(Hq + H) * d].unflatten(-1, (H, d))
        V = packed[..., (Hq + H) * d:].unflatten(-1, (H, d))
        pos = (torch.tensor(lens)[:, None] + torch.arange(L)).to(torch.int32).cuda()
        q, k = gb.qk_norm_rope(Q, K, gamma_q=gam, gamma_k=gam, rope=rope, positions=pos)
        for got, x in ((q, Q), (k, K)):
            ref = norm_rope(x.double(), gam.double(), pos, w, "half")
            assert float((got.double() - ref).abs().max()) <= half_step(torch.bfloat16) * float(ref.abs().max()) * 1.01
        gb.cache8_append(cache, k, V, ints(*lens), ints(*new))
        for b in range(B):
            for h in range(H):
                held[b][h].append(k[b, :new[b], h], V[b, :new[b], h])
                want = held[b][h].held()
                got = cache_rows(cache, b, h, lens[b] + new[b])
                assert all(torch.equal(x.cpu(), y) for x, y in zip(got, want)), (step, b, h)
        if L <= 128 // G:
            X, W = gate_inputs("elementwise", B, L, Hq, d, dm, 95 + step)
            O = gb.gated_sdpa_cache8(X, q, cache, ints(*lens), W, n_new=ints(*new))
            check_attention(O, X, q, cache, W, "elementwise", lens, new)
        lens = [a + n for a, n in zip(lens, new)]


def test_a_training_step_together():
    # norm and rotary positions -> gated attention -> its backward -> theirs, against autograd in 64 bits
    B, L, Hq, H, d, dm = 1, 150, 8, 4, 128, 128
    g = torch.Generator().manual_seed(99)
    Q, K, V = (torch.randn(B, L, n, d, generator=g).bfloat16().cuda() for n in (Hq, H, H))
    X = torch.randn(B, L, dm, generator=g).bfloat16().cuda()
    W = (torch.randn(dm, Hq * d, generator=g) / math.sqrt(dm)).bfloat16().cuda()
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    dO = torch.randn(B, L, Hq, d, generator=g).bfloat16().cuda()
    rope, w = gb.Rope(128), frequencies(128)
    kw = dict(gamma_q=gq, gamma_k=gk, rope=rope)
    q, k = gb.qk_norm_rope(Q, K, **kw)
    O, _, lse = gb.gated_sdpa_fwd_train(X, q, k, V, W)
    inner = gb.gated_sdpa_bwd(X, q, k, V, W, O, dO, lse)
    outer = gb.qk_norm_rope_bwd(Q, K, inner["dQ"], inner["dK"], **kw)

    pos = torch.arange(L, device="cuda").expand(B, L)
    leaves = {n: t.double().requires_grad_() for n, t in
              (("Q", Q), ("K", K), ("V", V), ("gq", gq), ("gk", gk), ("W", W))}
    q6 = norm_rope(leaves["Q"], leaves["gq"], pos, w, "half")
    k6 = norm_rope(leaves["K"], leaves["gk"], pos, w, "half").repeat_interleave(Hq // H, 2)
    v6 = leaves["V"].repeat_interleave(Hq // H, 2)
    s = torch.einsum("bihd,bjhd->bhij", q6, k6) / math.sqrt(d)
    s = s.masked_fill(torch.ones(L, L, device="cuda").triu(1).bool(), -math.inf)
    y = torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), v6)
    (y * torch.sigmoid(X.double() @ leaves["W"]).view(B, L, Hq, d)).backward(dO.double())
    # bf16 at each hand-over: q, k, O, the weights, dS, dQ and dK, 2^-8 relative each and of random sign;
    # eight of them in a row, none correlated, give a 2-norm of at most 8 * 2^-8 of the gradient's
    for got, ref in ((outer["dQ"], leaves["Q"]), (outer["dK"], leaves["K"]), (outer["dgamma_q"], leaves["gq"]),
                     (outer["dgamma_k"], leaves["gk"]), (inner["dV"], leaves["V"]), (inner["dW_g"], leaves["W"])):
        off = float((got.double() - ref.grad).norm() / ref.grad.norm())
        assert off <= 8 * half_step(torch.bfloat16)
