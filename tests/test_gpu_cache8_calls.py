"""Calls on the 8-bit cache as programs mix them: two threads on one stream, errors of
two kinds at once, lengths and capacities on both sides of where the kernels change
their way of working."""
import math
import threading

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from ops_ref import cache_rows

pytestmark = pytest.mark.gpu


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


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def filled_cache(lens, H, d, kind, seed, capacity=None):
    B, L = len(lens), max(1, max(lens))
    cache = gb.cache8_alloc(B, capacity or L, H, d, kind)
    gb.cache8_append(cache, randn(seed, B, L, H, d), randn(seed + 1, B, L, H, d), ints(*[0] * B), ints(*lens))
    return cache


def test_two_threads_on_one_stream():
    # heads cut between teams: each call's second kernel merges what its first left in the workspace
    work = []
    for k in range(2):
        lens = [5000 + 700 * k, 300]
        cache = filled_cache(lens, 2, 128, "int8", 10 + k)
        Q, at = randn(20 + k, 2, 1, 8, 128), ints(*[n - 1 for n in lens])
        X, W = randn(30 + k, 2, 1, 256), randn(40 + k, 256, 8) / 16
        x, dx = randn(50 + k, 1, 300, 6, 128), randn(60 + k, 1, 300, 6, 128)
        rope = gb.Rope(128)
        kv = [t[:, :, :2].contiguous() for t in (x, dx)]

        def call(cache=cache, Q=Q, at=at, X=X, W=W, x=x, dx=dx, rope=rope, kv=kv):
            grads = gb.qk_norm_rope_bwd(x, kv[0], dx, kv[1], rope=rope)
            return [gb.gated_sdpa_cache8(X, Q, cache, at, W, gate="headwise"), *grads.values()]
        work.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(2)

    def many(call, want):
        torch.cuda.set_device(0)
        start.wait()
        got = [call() for _ in range(200)]
        torch.cuda.synchronize()
        wrong.append(sum(not torch.equal(a, b) for g in got for a, b in zip(g, want)))
    threads = [threading.Thread(target=many, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


def test_a_timeout_and_a_length_out_of_range_are_both_reported():
    cache = filled_cache([64], 1, 64, "int8", 1)
    K = randn(2, 1, 1, 1, 64)
    for first in (0, 1):
        for step in (first, 1 - first):
            if step:
                gb.cache8_append(cache, K, K, ints(64))
            else:
                gb.set_wait_limit_ns(200_000)
                try:
                    assert gb.wait_self_test() == gb.OK      # a wait that nothing completes
                finally:
                    gb.set_wait_limit_ns(0)
        assert [gb.check_device_error() for _ in range(3)] == [gb.ERR_DEVICE_TIMEOUT, gb.ERR_CACHE_RANGE, gb.OK]
    gb.cache8_append(cache, K, K, ints(-1))
    assert [gb.check_device_error() for _ in range(2)] == [gb.ERR_CACHE_RANGE, gb.OK]


# ---------------------------------------------------------------- the attention to the kernel's own bound
def check(O, X, Q, cache, W, gate, lens, new, sequences=None):
    """Every row against the formula in 64 bits. With A the sum of weights times |v| over full blocks and A' over the
    open one, the output is off by at most 2^-11 A (weights rounded to fp16) + 2^-17 A' (two bf16 parts) + 2^-37 of
    the largest product of a weight and a value scale for each unit of a code (fp16's range) + twice the scores'
    error (d additions of 2^-23) and 2^-13 (additions of the weights, exponentials, the gate's sigmoid) of A + A';
    then it is rounded to bf16."""
    B, Lq, Hq, d = Q.shape
    H, G = cache.H_kv, Hq // cache.H_kv
    for b in range(B) if sequences is None else sequences:
        T, n = lens[b] + new[b], new[b]
        assert not bool(O[b, n:].any()), f"rows past n_new of sequence {b} are not zero"
        if n == 0:
            continue
        full, rest = T // 64, T % 64
        sig = torch.ones(n, Hq, d, dtype=torch.float64, device="cuda")
        if gate != "none":
            s = torch.sigmoid(X[b, :n].double() @ W.double())
            sig = s[..., None].expand(-1, -1, d) if gate == "headwise" else s.view(n, Hq, d)
        codes = cache.v8[b, :, :full].double().transpose(-1, -2).reshape(H, -1, d)
        scale = cache.v_scale[b, :, :full].double()
        k = (cache.k8[b, :, :full].double() * cache.k_scale[b, :, :full, None, None].double()).reshape(H, -1, d)
        k = torch.cat((k, cache.k_tail[b, :, full % 2, :rest].double()), 1)
        v = torch.cat((codes * scale.repeat_interleave(64, 1)[..., None],
                       cache.v_tail[b, :, full % 2, :, :rest].double().transpose(-1, -2)), 1)
        q = Q[b, :n].double().view(n, H, G, d).permute(1, 0, 2, 3).reshape(H, n * G, d)
        seen = torch.arange(T, device="cuda") <= lens[b] + torch.arange(n, device="cuda").repeat_interleave(G)[:, None]
        score = (q @ k.transpose(1, 2) / math.sqrt(d)).masked_fill(~seen, -math.inf)
        top = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1, keepdim=True) / math.sqrt(d)
        w = torch.softmax(score, -1)
        ref = w @ v
        closed, opened = w[..., :64 * full] @ v[:, :64 * full].abs(), w[..., 64 * full:] @ v[:, 64 * full:].abs()
        tol = (2.0 ** -11 * closed + 2.0 ** -17 * opened + (2 * d * 2.0 ** -23 * top + 2.0 ** -13) * (closed + opened))
        if full:
            tol = tol + 2.0 ** -37 * w.amax(-1, keepdim=True) * scale.amax(1)[:, None, None] * codes.abs().sum(1)[:, None]

        def rows(t):
            return t.view(H, n, G, d).permute(1, 0, 2, 3).reshape(n, Hq, d) * sig
        ref, tol = rows(ref), rows(tol) + 2.0 ** -8 * rows(ref).abs() + 1e-30
        err = (O[b, :n].double() - ref).abs()
        assert bool((err <= tol).all()), (b, T, float((err / tol).max()))


def run(cache, lens, new, G, Lq, gate, seed, sequences=None):
    B, H, d = len(lens), cache.H_kv, cache.d_k
    Q = randn(seed, B, Lq, H * G, d)
    X = W = None
    if gate != "none":
        X, W = randn(seed + 1, B, Lq, 256), randn(seed + 2, 256, H * G * (1 if gate == "headwise" else d)) / 16
    n = None if new == [Lq] * B else ints(*new)
    O = gb.gated_sdpa_cache8(X, Q, cache, ints(*lens), W, gate=gate, n_new=n)
    check(O, X, Q, cache, W, gate, lens, new, sequences)
    return O


@pytest.mark.parametrize("kind,gate", [("int8", "none"), ("e4m3", "headwise"), ("int8", "elementwise")])
@pytest.mark.parametrize("d,H,G,Lq", [(128, 2, 4, 1), (64, 1, 8, 1), (128, 8, 3, 5), (64, 2, 8, 4), (128, 1, 16, 8), (64, 1, 1, 70)])
@pytest.mark.parametrize("T", [64, 960, 3000])
def test_attention_to_its_bound(T, d, H, G, Lq, kind, gate):
    # full blocks alone, and an open block beside them, for each number of query rows
    if gate == "headwise" and H * G % 8:
        gate = "elementwise"
    T = max(T, 128 if Lq > 64 else T)
    lens_after, new = [T, T + 37, T - 5], [Lq, Lq, Lq // 2]
    cache = filled_cache(lens_after, H, d, kind, 3)
    run(cache, [a - n for a, n in zip(lens_after, new)], new, G, Lq, gate, 5)


@pytest.mark.parametrize("gate", ["none", "headwise"])
@pytest.mark.parametrize("G,Lq", [(4, 1), (16, 1), (8, 4), (8, 8), (32, 4)])
@pytest.mark.parametrize("T", [1, 63, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1024])
def test_short_sequences_in_a_long_cache(T, G, Lq, gate):
    # a head is one block of threads' where all have at most a tile for each of its teams (8, 4, 2 or 1 by the
    # number of query rows): lengths on both sides, in a cache for far more, an empty sequence beside them
    if T < Lq:
        Lq = 1
    lens_after, new = [T, 0, max(T - 7, 0)], [Lq, 0, min(Lq, max(T - 7, 0))]
    cache = filled_cache(lens_after, 2, 128, "int8", 6, capacity=64 * 1024)
    run(cache, [a - n for a, n in zip(lens_after, new)], new, G, Lq, gate, 7)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("G,Lq,blocks", [(4, 1, 24), (4, 1, 25), (12, 1, 24), (12, 1, 25), (8, 4, 12), (8, 4, 13), (8, 8, 6), (8, 8, 7),
                                         (32, 4, 3), (32, 4, 4)])
def test_capacities_that_choose_one_launch_or_two(kind, G, Lq, blocks):
    # three tiles for each team of a head's one block of threads, by the capacity: full, almost, and nearly empty
    T = 64 * blocks
    for lens_after in ([T, T - 1], [T - 64, 65], [9, 200]):
        lens_after = [min(x, T) for x in lens_after]
        cache = filled_cache(lens_after, 2, 64, kind, 8, capacity=T)
        new = [min(Lq, x) for x in lens_after]
        run(cache, [a - n for a, n in zip(lens_after, new)], new, G, Lq, "none", 9)


def test_many_short_sequences_by_the_length_and_by_the_place():
    # as many heads as there are blocks of threads and one more (152 multiprocessors): from there on heads are not
    # one block's each, whatever their length
    for B in (75, 76, 77, 80):
        lens_after = [1 + 37 * b % 500 for b in range(B)]
        cache = filled_cache(lens_after, 2, 64, "e4m3", 10, capacity=8192)
        run(cache, [n - 1 for n in lens_after], [1] * B, 4, 1, "none", 11)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_drafts_taken_back_again_and_again(kind):
    # steps of up to 90 tokens, and lengths taken back by anything that stays within 64 of the longest so far: the
    # cache is that of the tokens that were kept, appended at once
    H, d, cap = 2, 64, 1024
    g = torch.Generator().manual_seed(13)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))
    for seed in range(6):
        cache, longest = gb.cache8_alloc(1, cap, H, d, kind), 0
        k = v = torch.zeros(1, 0, H, d, device="cuda", dtype=torch.bfloat16)
        for step in range(40):
            n = min(pick(1, 90) if step % 3 == 0 else pick(1, 6), cap - k.shape[1])
            new = [randn(100 * step + 10 * seed + i, 1, n, H, d) for i in range(2)]
            gb.cache8_append(cache, *new, ints(k.shape[1]))
            k, v = torch.cat((k, new[0]), 1), torch.cat((v, new[1]), 1)
            longest = max(longest, k.shape[1])
            T = pick(max(longest - 64, 0), k.shape[1]) if longest < cap - 90 else k.shape[1]
            k, v = k[:, :T], v[:, :T]
            want = gb.cache8_alloc(1, cap, H, d, kind)
            gb.cache8_append(want, k.contiguous(), v.contiguous(), ints(0))
            for h in range(H):
                for x, y in zip(cache_rows(cache, 0, h, T), cache_rows(want, 0, h, T)):
                    assert torch.equal(x, y), (seed, step, T, longest)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_cache_of_more_than_32_bits_of_bytes(kind):
    # 4.6 GB each of keys and values: the last sequences' blocks, scales, open blocks and rows lie past 2^32 bytes
    B, H, d, cap = 1100, 8, 128, 4096
    lens_after = [0] * B
    for b, n in ((0, 130), (549, 64), (1097, 200), (1098, 1), (1099, 199)):
        lens_after[b] = n
    cache = gb.cache8_alloc(B, cap, H, d, kind)
    assert cache.k8.numel() > 2 ** 32
    K, V = randn(14, B, 200, H, d), randn(15, B, 200, H, d)
    gb.cache8_append(cache, K, V, ints(*[0] * B), ints(*lens_after))
    for b in (0, 1097, 1099):
        want = gb.cache8_alloc(1, cap, H, d, kind)
        gb.cache8_append(want, K[b:b + 1].contiguous(), V[b:b + 1].contiguous(), ints(0), ints(lens_after[b]))
        for h in (0, H - 1):
            for x, y in zip(cache_rows(cache, b, h, lens_after[b]), cache_rows(want, 0, h, lens_after[b])):
                assert torch.equal(x, y)
    new = [min(1, n) for n in lens_after]
    run(cache, [n - m for n, m in zip(lens_after, new)], new, 4, 1, "headwise", 16, [0, 5, 549, 1096, 1097, 1098, 1099])
    del cache, K, V
    torch.cuda.empty_cache()


def test_one_sequence_of_more_than_32_bits_of_bytes():
    # one head, 2^26 tokens of 64 columns: 4.3 GB each; every key but a few is zero, so the weights are known
    d, T = 64, 2 ** 26 + 64
    cache = gb.cache8_alloc(1, T, 1, d, "int8")
    for t in (cache.k8, cache.v8, cache.k_scale, cache.v_scale):
        t.zero_()
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    last = T // 64 - 1
    cache.k8[0, 0, last, 63, 0] = 100          # the last token: 100 q / sqrt(d) = 25 above the others, e^25 = 7.2e10
    cache.v8[0, 0, last, :, 63] = 3
    cache.v8[0, 0, 5, :, 7] = 1                # and one far from it, of weight e^-25
    Q = torch.zeros(1, 1, 4, d, device="cuda", dtype=torch.bfloat16)
    Q[..., 0] = 2.0
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(T - 1), gate="none")
    w = 1 / (1 + (T - 1) * math.exp(-25.0))
    assert float((O.double() - 3 * w).abs().max()) <= 2.0 ** -8 * 3
    O = gb.gated_sdpa_cache8(None, Q, cache, ints(T - 65), gate="none")      # without the last block: even weights
    assert float((O.double() * (T - 64) - 1).abs().max()) <= 2.0 ** -7
    del cache
    torch.cuda.empty_cache()
