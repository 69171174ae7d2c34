"""The attention over the 8-bit cache when its bounded waits run out: whoever gives
up, the copies of a CTA land before it ends, the status is reported and the next
call is right."""
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
def default_limit():
    gb.set_wait_limit_ns(0)
    yield
    gb.set_wait_limit_ns(0)
    assert gb.check_device_error() == gb.OK


def filled_cache(lens, H, d, kind, seed, capacity=None):
    B, g = len(lens), torch.Generator(device="cuda").manual_seed(seed)
    cache = gb.cache8_alloc(B, capacity or max(lens), H, d, kind)
    K, V = (torch.randn(B, max(lens), H, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    gb.cache8_append(cache, K, V, torch.zeros(B, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return cache


def with_a_tiny_limit(call):
    """The status of one call whose waits may last 1 ns."""
    gb.set_wait_limit_ns(1)
    try:
        call()
        return gb.check_device_error()
    finally:
        gb.set_wait_limit_ns(0)


# shares that their rings hold whole, with and without an open block: one tile to a team, a few, one
# CTA to a head, and teams of several warps
@pytest.mark.parametrize("lens,H,Hq,d,Lq", [([64], 1, 4, 128, 1), ([700, 64 * 16, 5], 2, 8, 128, 1), ([30000], 2, 8, 64, 1),
                                            ([400, 64], 2, 16, 128, 5), ([900], 1, 16, 64, 8)])
def test_shares_shorter_than_their_ring_give_up_cleanly(lens, H, Hq, d, Lq):
    cache = filled_cache(lens, H, d, "int8", 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    Q = torch.randn(len(lens), Lq, Hq, d, generator=g, device="cuda").bfloat16()
    at = torch.tensor([max(n - Lq, 0) for n in lens], dtype=torch.int32, device="cuda")
    call = lambda: gb.gated_sdpa_cache8(None, Q, cache, at, gate="none")  # noqa: E731
    want = call()
    for _ in range(10):
        assert with_a_tiny_limit(call) in (gb.OK, gb.ERR_DEVICE_TIMEOUT)
        assert torch.equal(call(), want) and gb.check_device_error() == gb.OK


@pytest.mark.parametrize("gate,dm", [("headwise", 64), ("headwise", 8192), ("elementwise", 256), ("elementwise", 8192)])
def test_gate_logits_give_up_cleanly(gate, dm):
    # few chunks of d_model, all copied at once, and many, whose products the epilogue waits for longest
    lens, H, Hq, d = [300, 64], 2, 8, 128
    cache = filled_cache(lens, H, d, "e4m3", 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    Q = torch.randn(2, 1, Hq, d, generator=g, device="cuda").bfloat16()
    X = torch.randn(2, 1, dm, generator=g, device="cuda").bfloat16()
    W = (torch.randn(dm, Hq if gate == "headwise" else Hq * d, generator=g, device="cuda") / dm ** 0.5).bfloat16()
    at = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    call = lambda: gb.gated_sdpa_cache8(X, Q, cache, at, W, gate=gate)  # noqa: E731
    want = call()
    for _ in range(10):
        assert with_a_tiny_limit(call) in (gb.OK, gb.ERR_DEVICE_TIMEOUT)
        assert torch.equal(call(), want) and gb.check_device_error() == gb.OK


def test_a_share_longer_than_its_ring_reports_the_timeout():
    # the copying warp finds its rings full until the first tiles have been used: with 1 ns it does not wait that long
    lens, H, Hq, d = [32768] * 8, 8, 32, 128
    cache = filled_cache(lens, H, d, "int8", 7)
    Q = torch.randn(8, 1, Hq, d, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    at = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    call = lambda: gb.gated_sdpa_cache8(None, Q, cache, at, gate="none")  # noqa: E731
    want = call()
    for _ in range(5):
        assert with_a_tiny_limit(call) == gb.ERR_DEVICE_TIMEOUT
        assert torch.equal(call(), want) and gb.check_device_error() == gb.OK
