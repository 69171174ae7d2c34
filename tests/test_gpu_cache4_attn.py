"""The gated attention over the paged 4-bit cache against the 64-bit formula on the
cache's own bytes, to the bound of the kernel's own roundings (check_attention)."""
import math
import random

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from cache4_ref import PAGE, check_attention, codes_and_scales, held, pages_of

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def filled(T, H, d, kind, seed, *, width=None, exp=-4, junk=0xFF, scale=None):
    """Requests of T tokens in pages that lie anywhere, everything else of the pool a byte that must not be
    used (0xFF: scales that are NaN); scale [tokens]: factors of the values."""
    need = [pages_of(t) for t in T]
    width = width or max(1, max(need))
    order = random.Random(seed).sample(range(sum(need) + 3), sum(need))
    table, at = torch.full((len(T), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cache = gb.cache4_alloc(sum(need) + 3, H, d, kind, k_exp=exp, v_exp=exp)
    cache.pool.fill_(junk)
    slots = torch.cat([table[b].long()[torch.arange(t) // PAGE] * PAGE + torch.arange(t) % PAGE for b, t in enumerate(T)]).cuda()
    N = len(slots)
    if N:
        V = randn(seed + 1, N, H, d)
        gb.cache4_append(cache, randn(seed, N, H, d), V if scale is None else (V * scale[:, None, None]).bfloat16(), slots)
    return cache, table.cuda()


def run(cache, table, T, new, G, gate, seed, *, most=None, more=0, q_scale=1.0, requests=None, granted=None):
    H, d = cache.H_kv, cache.d_k
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    N = cu[-1] + more
    Q = (randn(seed, N, H * G, d) * q_scale).bfloat16()
    X = W = None
    if gate != "none":
        X, W = randn(seed + 1, N, 256), randn(seed + 2, 256, H * G * (1 if gate == "headwise" else d)) / 16
    lens = [t - n for t, n in zip(T, new)]
    O = torch.full((N, H * G, d), 7.0, dtype=torch.bfloat16, device="cuda")
    gb.gated_sdpa_cache4(X, Q, cache, table, ints(lens), ints(cu), W, gate=gate, max_new=most or max(1, max(new)), out=O)
    check_attention(O, X, Q, cache, table, lens, new, cu, W, gate, requests)
    return Q, O


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gate", ["none", "headwise", "elementwise"])
@pytest.mark.parametrize("d,H,G", [(128, 2, 4), (64, 1, 8), (128, 1, 1), (64, 8, 2), (128, 1, 16), (64, 2, 12), (128, 5, 7)])
def test_one_token(d, H, G, gate, kind):
    if gate == "headwise" and H * G % 8:
        gate = "elementwise"
    T = [1, 2, 63, 64, 65, 127, 128, 129, 700, 1000, 2049]
    cache, table = filled(T, H, d, kind, 1)
    run(cache, table, T, [1] * len(T), G, gate, 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,H,G,most", [(128, 2, 4, 5), (64, 16, 1, 5), (128, 1, 8, 16), (64, 2, 7, 8), (64, 1, 1, 128), (128, 1, 1, 70),
                                        (128, 2, 16, 8), (64, 1, 128, 1), (128, 3, 3, 3)])
def test_drafts_and_short_pieces(d, H, G, most, kind):
    # one to many rows of a request, some with none, the first rows of a request, pieces across a page's end
    new = [most, 1, 0, max(1, most // 2), most, max(1, most - 1), most]
    T = [n + x for n, x in zip(new, [0, 63, 10, 64, 500, 1, 1999])]
    cache, table = filled(T, H, d, kind, 4)
    run(cache, table, T, new, G, "elementwise", 5, more=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,most", [(4, 1), (16, 1), (8, 4), (8, 8), (32, 4)])
@pytest.mark.parametrize("T", [1, 63, 64, 128, 129, 255, 257, 511, 513, 1024, 1025])
def test_short_requests_in_a_wide_table(T, G, most, kind):
    # a head is one block of threads' where all have at most a page for each of its teams (8, 4, 2 or 1 by the
    # number of query rows): lengths on both sides, in a table for far more, an empty request beside them
    if T < most:
        most = 1
    lengths, new = [T, 0, max(T - 7, 0)], [most, 0, min(most, max(T - 7, 0))]
    cache, table = filled(lengths, 2, 128, kind, 6, width=1024)
    run(cache, table, lengths, new, G, "headwise", 7, most=most)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,most,width", [(4, 1, 48), (4, 1, 49), (8, 1, 48), (8, 1, 49), (4, 1, 24), (4, 1, 25), (12, 1, 24), (12, 1, 25), (8, 4, 12), (8, 4, 13), (8, 8, 6),
                                          (8, 8, 7), (32, 4, 3), (32, 4, 4)])
def test_widths_that_choose_one_launch_or_two(G, most, width, kind):
    T = PAGE * width
    for lengths in ([T, T - 1], [T - 64, 65], [9, 200]):
        lengths = [min(x, T) for x in lengths]
        cache, table = filled(lengths, 2, 64, kind, 8, width=width)
        run(cache, table, lengths, [min(most, x) for x in lengths], G, "none", 9, most=most)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width", [47, 64, 65, 700])
@pytest.mark.parametrize("B", [37, 50, 51, 75, 76, 152, 153])
def test_numbers_of_heads_that_choose_one_block_for_each(B, width, kind):
    # heads of up to four pages to a team are one block of threads' where there are enough of them, by the table's width or
    # by the lengths: all alike, and as different as can be
    most = PAGE * min(width, 64)
    for T in ([most] * B, [most if b % 3 else 1 + 41 * b % most for b in range(B)], [most if b == B // 2 else 70 for b in range(B)]):
        cache, table = filled(T, 1, 64, kind, 60, width=width)
        run(cache, table, T, [1] * B, 4, "elementwise" if B % 2 else "none", 61, requests=sorted({0, 1, B // 2, B - 1, *range(3, B, 11)}))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_many_requests(d, kind):
    # more than the schedule looks up one by one, and as many heads as there are blocks of threads and one more
    for B in (75, 77, 129, 300):
        T = [1 + 37 * b % 500 for b in range(B)]
        cache, table = filled(T, 2, d, kind, 10, width=128)
        run(cache, table, T, [1] * B, 4, "none", 11)


@pytest.mark.parametrize("G", [2, 20])
@pytest.mark.parametrize("B", [1000, 8200])
def test_thousands_of_requests(B, G):
    # several to a place of the schedule's lookup, most of them of a page or none
    r = random.Random(B)
    T = [r.choice([0, 1, 30, 64, 65, r.randint(1, 200), 900 if b % 97 == 5 else 2]) for b in range(B)]
    cache, table = filled(T, 1, 64, "e2m1", 70, width=15)
    run(cache, table, T, [min(t, 1) for t in T], G, "none", 71, requests=sorted({0, B // 2, B - 1, *r.sample(range(B), 40), *range(5, B, 970)}))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,most", [(1, 3), (2, 2), (3, 1), (5, 1), (1, 4), (1, 5), (4, 2), (9, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_numbers_of_query_rows_on_both_sides_of_a_change(d, G, most, kind):
    # up to 4, 8 and 16 rows a K/V head's products are laid out in another way
    T = [most, 70, 333, 1500, 5000]
    cache, table = filled(T, 2, d, kind, 50)
    run(cache, table, T, [most] * 4 + [1], G, "elementwise", 51, most=most)


@pytest.mark.parametrize("G,most", [(4, 1), (8, 1), (8, 2), (16, 4), (16, 8)])
def test_more_heads_than_teams(G, most):
    # the merge goes by the places where shares begin; heads of no, one and several pages
    B, H = 330, 8
    T = [(53 * b) % 300 + most if b % 7 else 0 for b in range(B)]
    cache, table = filled(T, H, 64, "e2m1", 52)
    run(cache, table, T, [most if t else 0 for t in T], G, "none", 53, most=most, requests=range(0, B, 5))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [[30000], [64 * 152 * 16 + 1], [40000, 17, 25000], [0, 90000, 0, 3000]])
def test_blocks_of_threads_within_one_head_and_across_two(T, kind):
    # a block whose share is all of one head leaves one part, others one for each team
    cache, table = filled(T, 1, 64, kind, 54)
    new = [min(2, t) for t in T]
    run(cache, table, T, new, 4, "none", 55, most=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("first", [65, 100, 128])
@pytest.mark.parametrize("H", [1, 3, 5])
@pytest.mark.parametrize("d", [64, 128])
def test_a_head_of_two_pages_that_one_team_has_whole(d, H, first, kind):
    # 64 rows, two teams to a block of threads: the first has both pages of a head, the second only the place after them
    for T in ([first, 1088], [1088, first], [first, 1088, first, 0, first, first]):
        cache, table = filled(T, H, d, kind, 56)
        run(cache, table, T, [min(8, t) for t in T], 8, "none", 57)


@pytest.mark.parametrize("G,most", [(4, 1), (8, 1), (12, 1), (8, 3), (8, 8), (16, 8)])
@pytest.mark.parametrize("T", [5, 64, 65, 200])
def test_one_live_request_among_more_than_there_are_blocks(T, G, most):
    # a captured step with room for many requests, in which one has rows
    for B, at in ((256, 100), (200, 0), (153, 152)):
        lengths = [T if b == at else 0 for b in range(B)]
        new = [min(most, T) if b == at else 0 for b in range(B)]
        cache, table = filled(lengths, 1, 64, "int4", 58, width=4)
        run(cache, table, lengths, new, G, "none", 59, most=most, more=2)


@pytest.mark.parametrize("G,most", [(4, 1), (8, 1), (12, 1), (8, 3), (8, 8)])
@pytest.mark.parametrize("B,H", [(64, 8), (200, 1), (300, 2)])
def test_a_step_in_which_no_request_has_rows(B, H, G, most):
    # nothing granted, or nothing brought, with more heads than blocks of threads: rows are zero, nothing is left in
    # the workspace, and what lies behind the arrays (numbers that a longer batch would have) is not taken for requests
    width, n_rows, behind = 40, B * most, 9000
    cache = gb.cache4_alloc(50, H, 64, "e2m1")
    cache.pool.zero_()
    Q = randn(62, n_rows, H * G, 64)
    table = torch.zeros(behind, width, dtype=torch.int32, device="cuda")
    lens, granted = ints([64 * b % 2000 + 5 for b in range(behind)]), ints([most] * behind)
    granted[:B] = 0
    full = torch.arange(behind, dtype=torch.int32, device="cuda") * most
    none = full - full[B]
    none[:B] = 0
    need = gb.cache4_workspace_bytes(cache, B, width, n_rows, most, H * G, gate="none")
    for cu, new in ((full, granted), (none, None)):
        workspace, O = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda"), torch.full_like(Q, 7.0)
        gb.gated_sdpa_cache4(None, Q, cache, table[:B], lens[:B], cu[:B + 1], gate="none", max_new=most,
                             n_new=None if new is None else new[:B], out=O, workspace=workspace)
        assert not bool(O.any()) and bool((workspace == 0x5A).all())


@pytest.mark.parametrize("kind", KINDS)
def test_long_requests_beside_short_ones(kind):
    T = [20000, 3, 64 * 100, 1, 777]
    cache, table = filled(T, 2, 128, kind, 12)
    run(cache, table, T, [1, 1, 2, 1, 3], 4, "headwise", 13)


@pytest.mark.parametrize("kind", KINDS)
def test_the_same_as_the_bf16_attention_on_what_is_read_back(kind):
    # the values that the cache holds, read back, through the library's bf16 attention
    H, d, G, T, n = 2, 128, 4, 333, 8
    cache, table = filled([T], H, d, kind, 14)
    Q = randn(15, n, H * G, d)
    pos = torch.arange(T, device="cuda")
    K, V = gb.cache4_read(cache, table[0].long()[pos // PAGE] * PAGE + pos % PAGE)
    X, W = randn(16, n, 256), randn(17, 256, H * G * d) / 16
    O = gb.gated_sdpa_cache4(X, Q, cache, table, ints([T - n]), ints([0, n]), W, max_new=n)
    want, _ = gb.gated_sdpa_fwd(X[None], Q[None], K[None], V[None], W, causal=True)
    # weights in bf16 there (2^-8 each) and in fp16 here, outputs in bf16, sums of |v| below 3
    assert float((O.double() - want[0].double()).abs().max()) <= (2 * 2.0 ** -8 + 2.0 ** -9) * 3


@pytest.mark.parametrize("kind", KINDS)
def test_what_lies_behind_a_request_is_not_seen(kind):
    # the same to the last bit whatever the rest of the last page, and of the pool, holds
    T, new = [1, 65, 100, 640, 1000], [1, 1, 3, 2, 3]
    got = []
    for junk in (0x00, 0xFF, 0x7E, 0x3C):
        cache, table = filled(T, 2, 128, kind, 18, junk=junk)
        got.append(run(cache, table, T, new, 4, "none", 19)[1])
    assert all(torch.equal(got[0], x) for x in got[1:])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_all_sizes(d, kind):
    # values whose scales go from the least to the largest, page by page and token by token, under sharp and
    # flat weights
    T, H, G = 64 * 12 + 5, 2, 4
    for case in range(3):
        n = torch.arange(T, device="cuda")
        e = {0: (n // PAGE) % 12, 1: n % 14, 2: torch.where(n == 70, 13, 0)}[case]
        cache, table = filled([T], H, d, kind, 20, exp=-2, scale=torch.exp2(e.double() - 4))
        for q_scale in (0.0, 1.0, 12.0):
            run(cache, table, [T], [2], G, "none", 21, q_scale=q_scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("share", [0.5, 0.99, 0.999, 0.9999])
@pytest.mark.parametrize("G", [4, 16])
def test_a_token_of_no_value_that_takes_most_of_the_weight(G, share, kind):
    # one token with zero values before, among or behind 8191 others, which share what is left
    T, d, H = 8192, 128, 1
    cache, table = filled([T], H, d, kind, 22)
    Q = torch.zeros(1, G, d, dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = 1.0
    apart = math.log(share / (1 - share) * (T - 1)) * math.sqrt(d)
    for at in (0, 3000, T - 1):
        K = torch.zeros(T, H, d, device="cuda", dtype=torch.bfloat16)
        V = randn(23, T, H, d)
        K[at, :, 0], V[at] = apart, 0
        pos = torch.arange(T, device="cuda")
        gb.cache4_append(cache, K, V, table[0].long()[pos // PAGE] * PAGE + pos % PAGE)
        O = gb.gated_sdpa_cache4(None, Q, cache, table, ints([T - 1]), ints([0, 1]), gate="none")
        check_attention(O, None, Q, cache, table, [T - 1], [1], [0, 1], None, "none")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,most", [(4, 1), (8, 1), (4, 3), (8, 4), (16, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_code_of_zero_takes_no_part(d, G, most, kind):
    # keys whose codes are zero where the query is 2^14 times what it is elsewhere, and a token whose codes are zero in
    # most columns under a scale of 256 beside values of 2^-6: neither may cost the others' sums their last bits
    H, T = 2, [64, 65, 200]
    cache, table = filled(T, H, d, kind, 90, exp=0)
    N = sum(T)
    K, V = randn(91, N, H, d), randn(92, N, H, d) * 2.0 ** -6
    K[..., :16] *= 8
    K[..., 0], K[..., 1] = 0, 8 * (7 if kind == "int4" else 6)
    at = 0
    for t in T:
        V[at + 5], at = 0, at + t
    for b in range(len(T)):
        V[sum(T[:b]) + 5, :, ::16] = 256 * (7 if kind == "int4" else 6)
    slots = torch.cat([table[b].long()[torch.arange(t, device="cuda") // PAGE] * PAGE + torch.arange(t, device="cuda") % PAGE
                       for b, t in enumerate(T)])
    gb.cache4_append(cache, K, V, slots)
    new, cu, lens = [most] * 3, [most * b for b in range(4)], [t - most for t in T]
    Q = randn(93, 3 * most, H * G, d)
    Q[..., 2:16] *= 2.0 ** -4
    Q[..., 0], Q[..., 1] = 2.0 ** 14, 0
    O = gb.gated_sdpa_cache4(None, Q, cache, table, ints(lens), ints(cu), gate="none", max_new=most)
    check_attention(O, None, Q, cache, table, lens, new, cu, None, "none", more=0.0)


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_queries(kind):
    # one token has all the weight; queries of 2^-100, 2^60 and zero
    T = [300, 300, 300]
    cache, table = filled(T, 2, 128, kind, 24)
    for q_scale in (0.0, 2.0 ** -100, 1e3):
        run(cache, table, T, [1, 2, 1], 4, "none", 25, q_scale=q_scale)
    Q = torch.full((3, 8, 128), 0.0, dtype=torch.bfloat16, device="cuda")
    Q[:, :, ::2] = 2.0 ** 60
    Q[1] = 2.0 ** -130
    O = gb.gated_sdpa_cache4(None, Q, cache, table, ints([299] * 3), ints([0, 1, 2, 3]), gate="none")
    assert bool(O.isfinite().all())


def check_one_token_has_all(cache, table, T, Q, O):
    """Scores so far apart that each row is its largest score's token: its values, which bf16 holds, to the last bit. Rows
    whose two largest scores are nearer to each other than the kernel's sums (see check_attention) may be off are left out."""
    d, G = cache.d_k, Q.shape[1] // cache.H_kv
    pos = torch.arange(T, device="cuda")
    k, v = held(cache, table[0].long()[pos // PAGE] * PAGE + pos % PAGE)
    _, _, ks, _ = codes_and_scales(cache.pool, table[0].long()[pos // PAGE] * PAGE + pos % PAGE, cache.kind)
    wide = k.abs() + (16 * ks.repeat_interleave(16, -1) * 2.0 ** cache.k_exp if cache.kind == "int4" else 0.0)
    k, v, wide = (x.repeat_interleave(G, 1) for x in (k, v, wide))                 # [T, Hq, d]
    scores, off = torch.einsum("hd,thd->ht", Q[0].double(), k), torch.einsum("hd,thd->ht", Q[0].double().abs(), wide).amax(-1)
    top = scores.topk(2, -1)
    sure = top.values[:, 0] - top.values[:, 1] > 2 * 2 * d * 2.0 ** -23 * off
    assert int(sure.sum()) * 2 > len(sure)
    want = v[top.indices[:, 0], torch.arange(len(sure), device="cuda")]
    assert torch.equal(O[0].double()[sure], want[sure]), (O[0].double() - want)[sure].abs().max()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [4, 8, 12])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_as_large_as_keys_are_small(d, G, kind):
    # products of 2^120 and 2^-64: scores are ordinary numbers, those of zero keys zero
    T, H = 300, 2
    cache, table = filled([T], H, d, kind, 80, exp=0)
    small = gb.Cache4(cache.pool, kind, k_exp=-64)
    for exp in (117, 118, 120, 124):
        Q = (randn(81, 1, H * G, d).double().clamp(-2, 2) * 2.0 ** exp).bfloat16()
        O = gb.gated_sdpa_cache4(None, Q, small, table, ints([T - 1]), ints([0, 1]), gate="none")
        check_one_token_has_all(small, table, T, Q, O)
    pos = torch.arange(T, device="cuda")
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    gb.cache4_append(cache, torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda"), randn(82, T, H, d), slots)
    O = gb.gated_sdpa_cache4(None, Q, small, table, ints([T - 1]), ints([0, 1]), gate="none")
    check_attention(O, None, Q, small, table, [T - 1], [1], [0, 1], None, "none")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [4, 8, 12])
@pytest.mark.parametrize("top", [2.0 ** 126, 2.0 ** 127, 1.984375 * 2.0 ** 127, 3.3895313892515355e38])
def test_the_largest_queries(top, G, kind):
    # up to bf16's largest number
    T, H, d = 300, 2, 64
    cache, table = filled([T], H, d, kind, 83, exp=0)
    small = gb.Cache4(cache.pool, kind, k_exp=-64)
    Q = randn(84, 1, H * G, d).double()
    Q = (Q / Q.abs().amax(-1, keepdim=True) * top).bfloat16()
    assert bool(Q.isfinite().all())
    O = gb.gated_sdpa_cache4(None, Q, small, table, ints([T - 1]), ints([0, 1]), gate="none")
    check_one_token_has_all(small, table, T, Q, O)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [4, 8, 12])
@pytest.mark.parametrize("exp,k_exp", [(59, 64), (70, 64), (120, 64), (124, 0), (100, 30)])
def test_scores_past_float32(exp, k_exp, G, kind):
    # on both sides of zero, and all of them below it; zero keys beside them
    T, H, d = 300, 2, 128
    cache, table = filled([T], H, d, kind, 85, exp=0)
    large = gb.Cache4(cache.pool, kind, k_exp=k_exp)
    call = lambda Q: gb.gated_sdpa_cache4(None, Q, large, table, ints([T - 1]), ints([0, 1]), gate="none")  # noqa: E731
    Q = (randn(86, 1, H * G, d).double().clamp(-3.5, 3.5) * 2.0 ** exp).bfloat16()
    check_one_token_has_all(large, table, T, Q, call(Q))
    pos = torch.arange(T, device="cuda")
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    K, V = -randn(87, T, H, d).abs() * 100, randn(88, T, H, d)
    gb.cache4_append(cache, K, V, slots)
    check_one_token_has_all(large, table, T, Q.abs(), call(Q.abs()))
    K[7] = 0
    gb.cache4_append(cache, K, V, slots)
    check_one_token_has_all(large, table, T, Q.abs(), call(Q.abs()))
    gb.cache4_append(cache, torch.zeros_like(K), V, slots)
    check_attention(call(Q), None, Q, large, table, [T - 1], [1], [0, 1], None, "none")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("k_exp,v_exp", [(-64, 64), (64, -64), (-30, 3), (10, -20)])
def test_exponents(k_exp, v_exp, kind):
    T, H, d, G = [200, 70], 2, 64, 4
    cache, table = filled(T, H, d, kind, 26, exp=0)
    scaled = gb.Cache4(cache.pool, kind, k_exp=k_exp, v_exp=v_exp)
    cu, lens, new = [0, 2, 3], [198, 69], [2, 1]
    Q = (randn(27, 3, H * G, d).double() * 2.0 ** -k_exp).bfloat16()
    O = gb.gated_sdpa_cache4(None, Q, scaled, table, ints(lens), ints(cu), gate="none", max_new=2)
    check_attention(O, None, Q, scaled, table, lens, new, cu, None, "none")


@pytest.mark.parametrize("kind", KINDS)
def test_nan_is_seen_by_who_may_see_it(kind):
    T, H, d, G = 200, 2, 64, 2
    cache, table = filled([T], H, d, kind, 28)
    n, cu = 4, [0, 4]
    Q = randn(29, n, H * G, d)
    call = lambda: gb.gated_sdpa_cache4(None, Q, cache, table, ints([T - n]), ints(cu), gate="none", max_new=n)  # noqa: E731
    want = call()
    K, V = randn(30, 1, H, d), randn(31, 1, H, d)
    K[0, 1, 5] = math.nan
    gb.cache4_append(cache, K, V, table[0, 3].long().view(1) * PAGE + (T - 2) % PAGE)      # row 2's own token
    O = call()
    assert bool(O[2:, 2:].isnan().all()) and not bool(O[:2].isnan().any()) and not bool(O[:, :2].isnan().any())
    assert torch.equal(O[:2], want[:2])
    Q[1, 0, 3] = math.inf                                                                 # a query: its own row alone
    O = call()
    assert bool(O[1, 0].isnan().all()) and not bool(O[0].isnan().any()) and not bool(O[1, 1].isnan().any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [-1, 2 ** 31 - 1, -2 ** 31, "past"])
def test_a_page_outside_the_pool(page, kind):
    # rows that see one of its tokens are NaN, all others as ever, and the error is reported
    T, H, d, G = [300, 1000, 64 * 30], 2, 128, 4
    cache, table = filled(T, H, d, kind, 32)
    new, cu, lens = [2, 1, 2], [0, 2, 3, 5], [298, 999, 64 * 30 - 2]
    Q = randn(33, 5, H * G, d)
    call = lambda: gb.gated_sdpa_cache4(None, Q, cache, table, ints(lens), ints(cu), gate="none", max_new=2)  # noqa: E731
    want = call()
    old = int(table[1, 9])
    table[1, 9] = cache.n_pages if page == "past" else page
    O = call()
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert bool(O[2].isnan().all()) and torch.equal(O[:2], want[:2]) and torch.equal(O[3:], want[3:])
    table[1, 9] = old
    assert torch.equal(call(), want)
    # behind the request's end nothing is looked up
    wide = torch.cat((table, torch.full((3, 4), -5, dtype=torch.int32, device="cuda")), 1)
    assert torch.equal(gb.gated_sdpa_cache4(None, Q, cache, wide, ints(lens), ints(cu), gate="none", max_new=2), want)
    # a page that only the second of a request's rows sees
    one = table[:1].clone()
    first = gb.gated_sdpa_cache4(None, Q[:2].contiguous(), cache, one, ints([255]), ints([0, 2]), gate="none", max_new=2)
    one[0, 4] = -1
    O = gb.gated_sdpa_cache4(None, Q[:2].contiguous(), cache, one, ints([255]), ints([0, 2]), gate="none", max_new=2)
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert torch.equal(O[0], first[0]) and bool(O[1].isnan().all())


@pytest.mark.parametrize("lens,cu,granted", [
    ([-1, 5, 5], [0, 1, 2, 3], None), ([500, 5, 5], [0, 1, 2, 3], None), ([2 ** 31 - 1, 5, 5], [0, 1, 2, 3], None),
    ([5, 5, 5], [0, 3, 4, 5], None), ([5, 5, 5], [0, 1, 2, 9], None), ([5, 5, 5], [0, 1, 0, 1], None),
    ([5, 5, 5], [0, 1, 2, 3], [2, 1, 1]), ([5, 5, 5], [0, 1, 2, 3], [-1, 1, 1])])
def test_numbers_out_of_range_give_zero_rows(lens, cu, granted):
    cache, table = filled([100, 100, 100], 1, 64, "int4", 34)
    Q = randn(35, 5, 4, 64)
    O = torch.full_like(Q, 7.0)
    gb.gated_sdpa_cache4(None, Q, cache, table, ints(lens), ints(cu), gate="none", max_new=2,
                         n_new=None if granted is None else ints(granted), out=O)
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    bad = [b for b in range(3) if not (0 <= cu[b] <= cu[b + 1] <= 5 and cu[b + 1] - cu[b] <= 2 and 0 <= lens[b] <= 120 and
                                       (granted is None or 0 <= granted[b] <= cu[b + 1] - cu[b]))]
    assert bad
    if cu == sorted(cu):
        for b in range(3):
            part = O[max(cu[b], 0):min(cu[b + 1], 5)]
            assert bool((part == 0).all()) if b in bad else bool(part.any(-1).all())


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_were_not_granted_and_padded_rows(kind):
    T, new = [300, 200, 70, 5], [2, 3, 1, 1]
    cache, table = filled(T, 2, 64, kind, 36)
    cu, lens = [0, 2, 5, 6, 7], [t - n for t, n in zip(T, new)]
    Q = randn(37, 12, 8, 64)
    X, W = randn(38, 12, 256), randn(39, 256, 8) / 16
    X[7:] = math.nan                                  # a padded batch's rows may hold anything
    Q[7:] = math.nan
    O = gb.gated_sdpa_cache4(X, Q, cache, table, ints(lens), ints(cu), W, gate="headwise", max_new=3)
    check_attention(O, X, Q, cache, table, lens, new, cu, W, "headwise")
    granted = [2, 0, 1, 0]
    part = gb.gated_sdpa_cache4(X, Q, cache, table, ints(lens), ints(cu), W, gate="headwise", max_new=3, n_new=ints(granted))
    assert torch.equal(part[[0, 1, 5]], O[[0, 1, 5]]) and not bool(part[[2, 3, 4, 6, 7, 8, 9, 10, 11]].any())
    none = gb.gated_sdpa_cache4(None, Q, cache, table, ints(lens), ints([0] * 5), gate="none")
    assert not bool(none.any())
    empty = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    none = gb.gated_sdpa_cache4(None, Q, cache, empty, empty[:, 0], ints([0]), gate="none")
    assert not bool(none.any()) and none.shape == Q.shape
    assert gb.gated_sdpa_cache4(None, Q[:0], cache, table, ints(lens), ints([0] * 5), gate="none").shape == (0, 8, 64)


@pytest.mark.parametrize("kind", KINDS)
def test_requests_that_share_pages(kind):
    # a common prefix: the same pages in several rows of the table
    T = [640, 640, 640]
    cache, table = filled(T, 2, 128, kind, 40)
    table[1, :7] = table[0, :7]
    table[2, :9] = table[0, :9]
    run(cache, table, T, [1, 2, 4], 4, "none", 41)


def test_no_call_depends_on_the_order_of_execution():
    cache, table = filled([5000, 300, 9000, 64], 2, 128, "e2m1", 42)
    Q = randn(43, 4, 8, 128)
    X, W = randn(44, 4, 256), randn(45, 256, 8 * 128) / 16
    args = (X, Q, cache, table, ints([4999, 299, 8999, 63]), ints([0, 1, 2, 3, 4]), W)
    want = gb.gated_sdpa_cache4(*args)
    assert all(torch.equal(gb.gated_sdpa_cache4(*args), want) for _ in range(50))


def test_argument_checks():
    cache, table = filled([100], 2, 64, "int4", 46)
    Q, lens, cu = randn(47, 1, 4, 64), ints([99]), ints([0, 1])
    X, W = randn(48, 1, 64), randn(49, 64, 4 * 64)
    call = gb.gated_sdpa_cache4
    for bad in (lambda: call(X, Q[:, :, :32], cache, table, lens, cu, W), lambda: call(X, Q.float(), cache, table, lens, cu, W),
                lambda: call(None, Q, cache, table, lens, cu, W), lambda: call(X, Q, cache, table, lens, cu),
                lambda: call(X, Q, cache, table.long(), lens, cu, W), lambda: call(X, Q, cache, table, lens, cu[:1], W),
                lambda: call(X, Q, cache, table[0], lens, cu, W), lambda: call(X, Q, cache, table, None, cu, W),
                lambda: call(X, Q, cache, table, lens, cu, W[:, :5]), lambda: call(X[:, :63], Q, cache, table, lens, cu, W),
                lambda: call(X, Q, cache, table, lens, cu, W, out=Q[:0]), lambda: call(X, Q, cache, table, lens.cpu(), cu, W),
                lambda: call(X, Q, cache, table, lens, cu, W, n_new=ints([1, 1]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gb.GsdpaError) as e:
        call(X, Q, cache, table, lens, cu, W, max_new=65)
    assert e.value.status == gb.ERR_UNSUPPORTED
    with pytest.raises(gb.GsdpaError) as e:
        call(X, Q, cache, table, lens, cu, W, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gb.ERR_WORKSPACE
