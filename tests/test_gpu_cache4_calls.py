"""The paged 4-bit cache as programs use it: the plan, norm with positions, append and
attention step after step, captured and replayed, on other streams, from two threads;
waits that run out; pools past 32 bits of bytes."""
import math
import random
import threading

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from cache4_ref import PAGE, check_attention, held, pages_of

pytestmark = pytest.mark.gpu
KINDS = ["int4", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    gb.load()


@pytest.fixture(autouse=True)
def no_device_error():
    gb.set_wait_limit_ns(0)
    yield
    gb.set_wait_limit_ns(0)
    assert gb.check_device_error() == gb.OK


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


class Server:
    """What a server holds: the pool, the block table, the free pages, the lengths."""

    def __init__(self, B, width, n_pages, H, d, kind):
        self.cache = gb.cache4_alloc(n_pages, H, d, kind, k_exp=-4, v_exp=-4)
        self.cache.pool.fill_(0xFF)
        self.table = ints([[-1] * width] * B)
        self.free, self.n_free = torch.randperm(n_pages, device="cuda").int(), ints([n_pages])
        self.lens = ints([0] * B)


def step(s, Q, K, V, X, W, new, rope, *, most, keep=None, gate="headwise"):
    """One layer's step as a program writes it. Returns the plan and the layer's output."""
    p = gb.pages_step(s.lens, new, s.table, s.free, s.n_free, len(Q), keep=keep)
    q, k = gb.qk_norm_rope(Q[None], K[None], rope=rope, positions=p.positions)
    gb.cache4_append(s.cache, k[0], V, p.slots)
    at = s.lens if keep is None else keep
    O = gb.gated_sdpa_cache4(X, q[0], s.cache, s.table, at, p.cu, W, gate=gate, max_new=most, n_new=p.granted)
    s.n_free = p.n_free
    s.lens = at + p.granted
    return p, q[0], k[0], O


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,H,G", [(128, 2, 4), (64, 4, 2)])
def test_a_serving_run(d, H, G, kind):
    # requests come, are prefilled in pieces, grow by single tokens and drafts, some of which go back, and end;
    # keys and values that the cache holds are those of the tokens that stayed, wherever they lie
    r, B, width, dm = random.Random(5), 6, 6, 256
    s, rope = Server(B, width, 10, H, d, kind), gb.Rope(d)
    W = randn(1, dm, H * G * d) / 16
    kept = [[] for _ in range(B)]       # each request's (k, v) rows as appended
    waited = 0
    for n in range(40):
        keep = [0 if r.random() < 0.08 else max(0, len(x) - r.choice([0, 0, 0, 1, 2])) for x in kept]
        new = [min(r.choice([1, 9, 30, 32]) if k == 0 else r.choice([0, 1, 1, 4, 16]), width * PAGE - k) for k in keep]
        N = sum(new) + 2
        Q, K, V, X = randn(100 * n + 2, N, H * G, d), randn(100 * n + 3, N, H, d), randn(100 * n + 4, N, H, d), randn(100 * n + 5, N, dm)
        p, q, k, O = step(s, Q, K, V, X, W, ints(new), rope, most=32, keep=ints(keep), gate="elementwise")
        granted, cu = p.granted.tolist(), p.cu.tolist()
        waited += granted != new
        for b in range(B):
            kept[b] = kept[b][:keep[b]] + [(k[cu[b] + i], V[cu[b] + i]) for i in range(granted[b])]
        assert s.lens.tolist() == [len(x) for x in kept]
        check_attention(O, X, q, s.cache, s.table, keep, granted, cu, W, "elementwise")
    assert waited, "the pool was never short"
    # every token that is held, against a cache into which it was written alone
    for b in range(B):
        if not kept[b]:
            continue
        T = len(kept[b])
        pos = torch.arange(T, device="cuda")
        one = gb.cache4_alloc(pages_of(T), H, d, kind, k_exp=-4, v_exp=-4)
        gb.cache4_append(one, torch.stack([x for x, _ in kept[b]]), torch.stack([x for _, x in kept[b]]), pos)
        for x, y in zip(held(s.cache, s.table[b].long()[pos // PAGE] * PAGE + pos % PAGE), held(one, pos)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_in_pieces(kind):
    # the pieces' own attention is the bf16 one, on what is read back of the pieces before and itself
    H, G, d, dm, T, piece = 2, 4, 128, 256, 700, 256
    s, rope, W = Server(1, 16, 20, H, d, kind), gb.Rope(d), randn(1, dm, H * G * d) / 16
    Q, K, V, X = randn(2, T, H * G, d), randn(3, T, H, d), randn(4, T, H, d), randn(5, T, dm)
    out = []
    for at in range(0, T, piece):
        n = min(piece, T - at)
        p = gb.pages_step(s.lens, ints([n]), s.table, s.free, s.n_free, n)
        q, k = gb.qk_norm_rope(Q[None, at:at + n], K[None, at:at + n], rope=rope, positions=p.positions)
        gb.cache4_append(s.cache, k[0], V[at:at + n], p.slots)
        pos = torch.arange(at + n, device="cuda")
        kk, vv = gb.cache4_read(s.cache, s.table[0].long()[pos // PAGE] * PAGE + pos % PAGE)
        out.append(gb.gated_sdpa_fwd(X[None, at:at + n], q, kk[None], vv[None], W)[0][0])
        s.n_free, s.lens = p.n_free, s.lens + p.granted
    q, _ = gb.qk_norm_rope(Q[None], K[None], rope=rope)
    whole, _ = gb.gated_sdpa_fwd(X[None], q, kk[None], vv[None], W)
    # weights and outputs rounded to bf16 in either, of sums of |v| below 3
    assert float((torch.cat(out).double() - whole[0].double()).abs().max()) <= (2 * 2.0 ** -8 + 2.0 ** -8) * 3
    # and a token after the prompt, by the cache's own attention
    x = randn(6, 1, dm)
    p, q, k, O = step(s, randn(7, 1, H * G, d), randn(8, 1, H, d), randn(9, 1, H, d), x, W, ints([1]), rope, most=1, gate="elementwise")
    check_attention(O, x, q, s.cache, s.table, [T], [1], [0, 1], W, "elementwise")


@pytest.mark.parametrize("kind", KINDS)
def test_a_captured_step(kind):
    # a decoding step captured once, everything of it in place: replayed it takes pages, writes and attends as the
    # calls do, from whatever lengths the device holds
    H, G, d, dm, B, width = 2, 4, 128, 256, 5, 8
    rope, W, new = gb.Rope(d), randn(1, dm, H * G) / 16, ints([1] * B)
    first = [0, 62, 63, 200, 319]

    def fresh():
        torch.manual_seed(3)
        s = Server(B, width, 40, H, d, kind)
        N = sum(first)
        p = gb.pages_step(s.lens, ints(first), s.table, s.free, s.n_free, N)
        gb.cache4_append(s.cache, randn(10, N, H, d), randn(11, N, H, d), p.slots)
        s.lens, s.n_free = s.lens + p.granted, p.n_free.clone()
        return s

    def inputs(i):
        return randn(20 + i, B, H * G, d), randn(40 + i, B, H, d), randn(60 + i, B, H, d), randn(80 + i, B, dm)
    s = fresh()
    want = [step(s, *inputs(i), W, new, rope, most=1)[3].clone() for i in range(6)]
    t = fresh()
    held_in = [torch.empty_like(x) for x in inputs(0)]

    def body():
        p = gb.pages_step(t.lens, new, t.table, t.free, t.n_free, B)
        q, k = gb.qk_norm_rope(held_in[0][None], held_in[1][None], rope=rope, positions=p.positions)
        gb.cache4_append(t.cache, k[0], held_in[2], p.slots)
        O = gb.gated_sdpa_cache4(held_in[3], q[0], t.cache, t.table, t.lens, p.cu, W, gate="headwise", n_new=p.granted)
        t.n_free.copy_(p.n_free)
        t.lens.add_(p.granted)
        return O
    for x, y in zip(held_in, inputs(0)):
        x.copy_(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            O = body()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(6):
        for x, y in zip(held_in, inputs(i)):
            x.copy_(y)
        graph.replay()
        assert torch.equal(O, want[i]), i
    assert t.lens.tolist() == s.lens.tolist() and t.n_free.tolist() == s.n_free.tolist() and torch.equal(t.table, s.table)


@pytest.mark.parametrize("Hq", [8, 24, 80])
def test_a_captured_call_for_other_lengths(Hq):
    # captured once for a wide table and replayed for lengths at which heads are one block's each, are cut, or are not there
    B, H, d, width = 6, 2, 64, 300
    s = Server(B, width, B * width, H, d, "int4")
    s.table.copy_(s.free.view(B, -1))
    pos = torch.arange(B * width * PAGE, device="cuda")
    gb.cache4_append(s.cache, randn(1, len(pos), H, d), randn(2, len(pos), H, d), pos)
    Q, lens, cu = randn(3, B, Hq, d), ints([0] * B), ints(list(range(B + 1)))
    call = lambda: gb.gated_sdpa_cache4(None, Q, s.cache, s.table, lens, cu, gate="none")  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = call()
    for T in ([1] * B, [64 * 15] * B, [1500, 40, 1, 700, 1500, 2], [width * PAGE] * B, [1, 1, 19000, 1, 1, 1], [5] * B,
              [4000, 9000, 0, 63, 64, 65], [64 * 31] * B):
        lens.copy_(ints([t - 1 for t in T]))
        O.fill_(7.0)
        graph.replay()
        assert torch.equal(O, call())
        if 0 not in T:
            check_attention(O, None, Q, s.cache, s.table, [t - 1 for t in T], [1] * B, list(range(B + 1)), None, "none")
            continue
        empty = T.index(0)        # (a length that is none, -1: a zero row, and the error)
        assert not bool(O[empty].any())
        assert gb.check_device_error() == gb.ERR_CACHE_RANGE


def test_two_captured_graphs_at_once():
    graphs = []
    for k in range(2):
        H, d, T = 2, 128, [6000 + 500 * k, 40]
        s = Server(2, 110, 220, H, d, "e2m1")
        p = gb.pages_step(s.lens, ints(T), s.table, s.free, s.n_free, sum(T))
        gb.cache4_append(s.cache, randn(1 + k, sum(T), H, d), randn(3 + k, sum(T), H, d), p.slots)
        Q, X, W = randn(5 + k, 2, 8, d), randn(7 + k, 2, 256), randn(9 + k, 256, 8) / 16
        args = (X, Q, s.cache, s.table, ints([t - 1 for t in T]), ints([0, 1, 2]), W)
        want = gb.gated_sdpa_cache4(*args, gate="headwise").clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [gb.gated_sdpa_cache4(*args, gate="headwise") for _ in range(3)]
        graphs.append((graph, out, want, torch.cuda.Stream(), s, args))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, out, _, stream, *_ in graphs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for graph, _, _, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, out, want, *_ in graphs for o in out)


def test_on_a_stream_that_is_given():
    H, d, T = 2, 64, 500
    s = Server(1, 8, 10, H, d, "int4")
    side = torch.cuda.Stream()
    K, V, Q = randn(1, T, H, d), randn(2, T, H, d), randn(3, 1, 8, d)
    torch.cuda.synchronize()
    p = gb.pages_step(s.lens, ints([T]), s.table, s.free, s.n_free, T, stream=side)
    gb.cache4_append(s.cache, K, V, p.slots, stream=side)
    at, cu = ints([T - 1]), ints([0, 1])
    side.wait_stream(torch.cuda.current_stream())
    O = gb.gated_sdpa_cache4(None, Q, s.cache, s.table, at, cu, gate="none", stream=side)
    k, v = gb.cache4_read(s.cache, p.slots, stream=side)
    side.synchronize()
    check_attention(O, None, Q, s.cache, s.table, [T - 1], [1], [0, 1], None, "none")
    want = held(s.cache, p.slots)
    assert torch.equal(k.double(), want[0]) and torch.equal(v.double(), want[1])


def test_two_threads_on_one_stream():
    work = []
    for n in range(2):
        H, d, T = 2, 128, [5000 + 700 * n, 300]
        s = Server(2, 100, 200, H, d, KINDS[n])
        p = gb.pages_step(s.lens, ints(T), s.table, s.free, s.n_free, sum(T))
        K, V = randn(1 + n, sum(T), H, d), randn(3 + n, sum(T), H, d)
        gb.cache4_append(s.cache, K, V, p.slots)
        Q, X, W = randn(5 + n, 2, 8, d), randn(7 + n, 2, 256), randn(9 + n, 256, 8) / 16
        at, cu = ints([t - 1 for t in T]), ints([0, 1, 2])

        def call(s=s, p=p, Q=Q, X=X, W=W, at=at, cu=cu, T=T, K=K, V=V):
            gb.cache4_append(s.cache, K[:64], V[:64], p.slots[:64])
            plan = gb.pages_step(at, ints([1, 1]), s.table, s.free, p.n_free, 2)
            return [gb.gated_sdpa_cache4(X, Q, s.cache, s.table, at, cu, W, gate="headwise"), plan.slots, *gb.cache4_read(s.cache, plan.slots)]
        work.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(2)

    def many(call, want):
        torch.cuda.set_device(0)
        begin.wait()
        got = [call() for _ in range(200)]
        torch.cuda.synchronize()
        wrong.append(sum(not torch.equal(a, b) for g in got for a, b in zip(g, want)))
    threads = [threading.Thread(target=many, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


def test_appends_at_once_to_one_tile():
    # two streams write the even and the odd tokens of the same pages: no byte is two tokens'
    H, d, N = 4, 128, 256
    for kind in KINDS:
        K, V, slots = randn(1, N, H, d), randn(2, N, H, d), torch.arange(N, device="cuda")
        want = gb.cache4_alloc(4, H, d, kind)
        gb.cache4_append(want, K, V, slots)
        parts = [[x[i::2].contiguous() for x in (K, V, slots)] for i in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(30):
            got = gb.cache4_alloc(4, H, d, kind)
            torch.cuda.synchronize()
            for part, stream in zip(parts, streams):
                gb.cache4_append(got, *part, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got.pool, want.pool)


# ---------------------------------------------------------------- waits that run out
def with_a_tiny_limit(call):
    """The status of one call whose waits may last 1 ns."""
    gb.set_wait_limit_ns(1)
    try:
        call()
        return gb.check_device_error()
    finally:
        gb.set_wait_limit_ns(0)


# shares that their rings hold whole: one tile to a team, a few, one CTA to a head, and teams of several warps; pages
# outside the pool, which no copy brings
@pytest.mark.parametrize("T,H,Hq,d,n,bad", [([64], 1, 4, 128, 1, False), ([700, 1024, 5], 2, 8, 128, 1, False),
                                            ([30000], 2, 8, 64, 1, False), ([400, 64], 2, 16, 128, 5, True),
                                            ([900], 1, 16, 64, 8, False), ([900, 64], 2, 8, 64, 1, True)])
def test_shares_shorter_than_their_ring_give_up_cleanly(T, H, Hq, d, n, bad):
    s = Server(len(T), pages_of(max(T)), sum(map(pages_of, T)), H, d, "int4")
    p = gb.pages_step(s.lens, ints(T), s.table, s.free, s.n_free, sum(T))
    gb.cache4_append(s.cache, randn(1, sum(T), H, d), randn(2, sum(T), H, d), p.slots)
    if bad:
        s.table[0, 0] = -1
    Q = randn(3, n * len(T), Hq, d)
    args = (None, Q, s.cache, s.table, ints([max(t - n, 0) for t in T]), ints([n * b for b in range(len(T) + 1)]))
    call = lambda: gb.gated_sdpa_cache4(*args, gate="none", max_new=n)  # noqa: E731
    want, fine = call(), gb.ERR_CACHE_RANGE if bad else gb.OK
    assert gb.check_device_error() == fine

    def same(x):
        return torch.equal(x.nan_to_num(nan=99.0), want.nan_to_num(nan=99.0))
    for _ in range(10):
        status = with_a_tiny_limit(call)
        assert status in (fine, gb.ERR_DEVICE_TIMEOUT)
        if bad and status != fine:
            assert gb.check_device_error() in (gb.OK, gb.ERR_CACHE_RANGE)
        assert same(call()) and gb.check_device_error() == fine


# up to 8 query rows a warp waits for its own copies only, which may be there before it looks at the time; with
# more a copying warp finds its rings full until the first tiles have been used, and with 1 ns does not wait that long
@pytest.mark.parametrize("Hq,certain", [(32, False), (128, True)])
def test_shares_longer_than_their_ring_give_up_cleanly(Hq, certain):
    B, T, H, d = 8, 32768, 8, 128
    s = Server(B, T // PAGE, B * T // PAGE, H, d, "e2m1")
    s.table.copy_(s.free.view(B, -1))
    s.cache.pool.copy_(torch.randint(0, 100, s.cache.pool.shape, device="cuda", dtype=torch.uint8))    # no scale is NaN
    args = (None, randn(1, B, Hq, d), s.cache, s.table, ints([T - 1] * B), ints(list(range(B + 1))))
    call = lambda: gb.gated_sdpa_cache4(*args, gate="none")  # noqa: E731
    want = call()
    for _ in range(5):
        status = with_a_tiny_limit(call)
        assert status == gb.ERR_DEVICE_TIMEOUT or (status == gb.OK and not certain)
        assert torch.equal(call(), want) and gb.check_device_error() == gb.OK


# ---------------------------------------------------------------- past 32 bits
def test_a_pool_of_more_than_32_bits_of_bytes():
    H, d, kind = 8, 128, "int4"
    n_pages = 2 ** 32 // (H * 72 * d) + 700
    cache = gb.cache4_alloc(n_pages, H, d, kind, k_exp=-4, v_exp=-4)
    T, width = [1000, 130, 64], 16
    table = torch.full((3, width), -1, dtype=torch.int32)
    table[0] = torch.arange(n_pages - 16, n_pages)
    table[1, :3] = torch.tensor([0, n_pages - 500, 3])
    table[2, 0] = n_pages - 20
    slots = torch.cat([table[b].long()[torch.arange(t) // PAGE] * PAGE + torch.arange(t) % PAGE for b, t in enumerate(T)]).cuda()
    gb.cache4_append(cache, randn(1, sum(T), H, d), randn(2, sum(T), H, d), slots)
    Q = randn(3, 3, 32, d)
    lens, cu = [t - 1 for t in T], [0, 1, 2, 3]
    O = gb.gated_sdpa_cache4(None, Q, cache, table.cuda(), ints(lens), ints(cu), gate="none")
    check_attention(O, None, Q, cache, table.cuda(), lens, [1] * 3, cu, None, "none")
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", KINDS)
def test_a_request_of_more_than_32_bits_of_bytes(kind):
    # one head, 2^26 tokens of 64 columns, 4.8 GB; every key but one has scale zero, so the weights are known
    d, T = 64, 2 ** 26 + 64
    n = T // PAGE
    cache = gb.cache4_alloc(n, 1, d, kind)
    cache.pool.zero_()
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    K, V = torch.zeros(2, 1, d, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 1, d, device="cuda", dtype=torch.bfloat16)
    K[0, 0, 0] = 112.0 if kind == "int4" else 96.0       # the last token: 25 or so above the others
    V[0], V[1] = 3.0, 1.0                                # and one far from it
    last, far = (0 * PAGE + 63), (n - 6) * PAGE + 7      # (the table is turned round)
    slots = torch.tensor([last, far], device="cuda")
    gb.cache4_append(cache, K, V, slots)
    k, v = held(cache, slots)
    key, high, low = float(k[0, 0, 0]), float(v[0, 0, 0]), float(v[1, 0, 0])
    Q = torch.zeros(1, 4, d, device="cuda", dtype=torch.bfloat16)
    Q[..., 0] = 2.0
    top = 2.0 * key / 8
    O = gb.gated_sdpa_cache4(None, Q, cache, table, ints([T - 1]), ints([0, 1]), gate="none")
    w = 1 / (1 + (T - 1) * math.exp(-top))
    assert float((O.double() - high * w).abs().max()) <= 2.0 ** -8 * high
    O = gb.gated_sdpa_cache4(None, Q, cache, table, ints([T - 65]), ints([0, 1]), gate="none")     # without the last page: even weights
    assert float((O.double() * (T - 64) - low).abs().max()) <= 2.0 ** -7 * low
    del cache
    torch.cuda.empty_cache()
