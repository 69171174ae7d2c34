"""The handles of the operators around the attention on the host: copies and pickles of
the rotary plan, of a cache's description."""
import copy
import ctypes
import pickle

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gb.load()


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))], ids=["copy", "deepcopy", "pickle"])
def test_a_copied_rope_points_to_its_own_plan(how):
    rope = gb.Rope(64, layout="interleaved", scaling="parts", factor=8.0, orig_len=4096)
    bits = bytes(rope.plan)
    other = how(rope)
    assert other.ref == ctypes.addressof(other.plan)
    assert other.plan is not rope.plan and other.ref != rope.ref
    del rope
    assert bytes(other.plan) == bits
    # as part of a model, twice: still one plan
    a, b = how([other, other])
    assert bytes(a.plan) == bits and a.ref == ctypes.addressof(a.plan) and a is b


def test_a_plan_of_another_size_is_refused():
    with pytest.raises(ValueError, match="bytes"):
        gb._rope_of(b"\0" * 8)


class _Tensors(gb.Cache8):
    """A Cache8 over host tensors, for the copies alone (no call takes it)."""

    def __init__(self, *tensors):
        self.k8, self.v8, self.k_scale, self.v_scale, self.k_tail, self.v_tail = tensors
        self.plan = gb._Cache8Plan(0, 1, 1, 64, 64, *(t.data_ptr() for t in tensors))
        self.ref = ctypes.addressof(self.plan)


def test_a_copied_cache_is_made_of_its_own_tensors(monkeypatch):
    monkeypatch.setattr(gb, "Cache8", _Tensors)
    c = _Tensors(*(torch.full((4,), float(k)) for k in range(6)))
    for other in (copy.deepcopy(c), pickle.loads(pickle.dumps([t for t in c.__reduce__()[1]]))):
        ts = other if isinstance(other, list) else [getattr(other, n) for n in ("k8", "v8", "k_scale", "v_scale", "k_tail", "v_tail")]
        for k, t in enumerate(ts):
            assert torch.equal(t, torch.full((4,), float(k)))
            assert t.data_ptr() != (c.k8, c.v8, c.k_scale, c.v_scale, c.k_tail, c.v_tail)[k].data_ptr()
        if other is not ts:
            assert other.ref == ctypes.addressof(other.plan) and other.plan.k8 == other.k8.data_ptr()
    same = copy.copy(c)      # a second handle over the same tensors
    assert same.k8 is c.k8 and same.ref == ctypes.addressof(same.plan) != c.ref and same.plan.k8 == c.k8.data_ptr()


# ---------------------------------------------------------------- kept workspaces
@pytest.fixture
def on_the_host(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch.device("cpu")


def in_a_thread(f):
    import threading
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join()
    return out[0]


def test_two_threads_on_one_stream_do_not_share_a_workspace(on_the_host):
    # a call is several kernels, and the library is called without the interpreter's lock: on one stream
    # another thread's kernels may come between them
    mine = gb._kept_workspace(256, on_the_host, 11)
    assert gb._kept_workspace(200, on_the_host, 11) is mine          # the next call of this thread
    assert gb._kept_workspace(256, on_the_host, 12) is not mine      # another stream
    other = in_a_thread(lambda: gb._kept_workspace(256, on_the_host, 11))
    assert other.data_ptr() != mine.data_ptr()
    assert gb._kept_workspace(256, on_the_host, 11) is mine
    assert gb._kept_workspace(512, on_the_host, 11).numel() == 512   # a larger one takes its place
    assert gb._kept_workspace(0, on_the_host, 11) is None


def test_kept_workspaces_are_released(on_the_host):
    import weakref
    ref = weakref.ref(gb._kept_workspace(256, on_the_host, 21))
    assert ref() is not None
    in_a_thread(gb.release_workspaces)                                # another thread's: not this one's
    assert gb._kept_workspace(256, on_the_host, 21) is ref()
    gb.release_workspaces()
    assert ref() is None
    gone = in_a_thread(lambda: weakref.ref(gb._kept_workspace(256, on_the_host, 21)))
    assert gone() is None                                             # a thread's end is as good
    assert gb._kept_workspace(64, on_the_host, 21).numel() == 64


# ---------------------------------------------------------------- the rotary plan's angles
def two_pi(bits):
    """2 pi as an integer, times 2^bits (Machin's formula: pi = 16 atan(1/5) - 4 atan(1/239))."""
    def atan_inverse(n):
        term = (1 << bits + 32) // n
        total, k, sign = term, 1, 1
        while term:
            term //= n * n
            k, sign = k + 2, -sign
            total += sign * (term // k)
        return total
    return 2 * (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 32


@pytest.mark.parametrize("w", [1.0, 0.75, 2.0 ** -40, -2.0 ** -40, 1e-9, -0.25, 7.0, -1000.5, 12345.678, 3e8, -2.5e15, 1e300, 0.0])
def test_frequencies_of_any_size_keep_their_angle(w):
    # turns per position modulo one, to the 64 bits that are kept: an angle at any 32-bit position is then off by
    # |p| 2^-62 turns at most
    from fractions import Fraction
    rope = gb.Rope(16, inv_freq=[w] * 8)
    want = Fraction(w) / Fraction(two_pi(1400), 1 << 1400)
    off = (Fraction(rope.plan.turn[3], 1 << 64) - want) % 1
    assert min(off, 1 - off) <= Fraction(1, 1 << 62) + abs(want) / (1 << 100)
