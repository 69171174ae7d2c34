"""Calls on the 8-bit cache as programs mix them: two threads on one stream, errors of
two kinds at once, lengths and capacities on both sides of where the kernels change
their way of working."""
import math
import threading

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild

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
