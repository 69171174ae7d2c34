"""The plan of a step over a paged cache against the plain one, number by number: growth,
pages given back, pools that do not suffice, padded batches, numbers out of range."""
import random

import pytest
import torch

from gated_softmax_attention_gb300 import binding as gb
from gated_softmax_attention_gb300 import build as gbuild
from cache4_ref import PAGE, pages_of, plan

pytestmark = pytest.mark.gpu


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


def start(lens, width, spare, seed):
    """A pool in use: the requests' pages and `spare` free ones, anywhere."""
    n = sum(map(pages_of, lens)) + spare
    order = random.Random(seed).sample(range(max(n, 1)), n)
    table, at = [], 0
    for x in lens:
        p = pages_of(x)
        table.append(order[at:at + p] + [-7] * (width - p))
        at += p
    return table, order[at:], max(n, 1)


def check(lens, new, width, spare, seed, keep=None, more=0, out=None):
    table, free, n_pages = start(lens, width, spare, seed)
    n_rows = sum(new) + more
    stack = ints(free + [-9] * (n_pages - len(free)))
    got_table, n_free = ints(table).view(len(lens), width), ints([len(free)])
    step = gb.pages_step(ints(lens), ints(new), got_table, stack, n_free, n_rows, keep=None if keep is None else ints(keep),
                         out=out)
    cu, granted, slots, positions, left, want_table, want_stack = plan(lens, new, table, free, len(free), n_rows, width, keep)
    assert step.cu.tolist() == cu and step.granted.tolist() == granted
    assert step.slots.tolist() == slots and step.positions.tolist() == positions
    assert step.n_free.tolist() == [left] and (out is not None or n_free.tolist() == [len(free)])
    assert got_table.tolist() == want_table
    assert stack.tolist()[:left] == want_stack[:left]
    return granted


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("B", [1, 2, 31, 33, 255, 256, 257, 1024, 1025, 3000, 8192])
def test_growth(B, seed):
    r = random.Random(seed)
    lens = [r.choice([0, 1, 63, 64, 65, 127, 128, r.randint(0, 700)]) for _ in range(B)]
    new = [r.choice([0, 1, 1, 1, 2, 64, 65, r.randint(0, 200) if B < 2000 else 1]) for _ in range(B)]
    need = sum(pages_of(a + b) - pages_of(a) for a, b in zip(lens, new))
    assert check(lens, new, 16, need, seed) == new                        # exactly enough
    if need:
        granted = check(lens, new, 16, need - 1, seed, more=r.choice([0, 1, 300]))
        assert granted != new                                             # the last that needs one goes without


@pytest.mark.parametrize("seed", range(12))
def test_pages_given_back_and_taken(seed):
    r = random.Random(100 + seed)
    B = r.choice([1, 5, 64, 300, 1500])
    lens = [r.randint(0, 900) for _ in range(B)]
    keep = [r.choice([x, x, 0, max(0, x - 1), max(0, x - 64), r.randint(0, x)]) for x in lens]
    new = [r.choice([0, 1, 5, 64, r.randint(0, 300)]) for _ in range(B)]
    check(lens, new, 24, r.choice([0, 1, 7, 3 * B]), seed, keep=keep)


def test_prompts_of_many_rows():
    # more rows than the planning block fills in itself: on both sides of where the second kernel takes them
    for new in ([2047], [2048], [2049], [0, 5000, 1, 0, 3, 9000, 0], [1] * 2000 + [64]):
        lens = [17 * k % 200 for k in range(len(new))]
        check(lens, new, 200, 400, 5, more=3)


@pytest.mark.parametrize("rows", [511, 512, 513, 2047, 2048, 2049])
@pytest.mark.parametrize("B", [1, 256, 257])
def test_rows_on_both_sides_of_the_second_kernel(B, rows):
    # two rows to a thread of the planning block, which has 256 or 1024
    new = [rows - (B - 1)] + [1] * (B - 1)
    check([17 * k % 200 for k in range(B)], new, 40, 400 + B, 6, more=0)


def test_in_place_and_written_again():
    # n_free in place, as a captured step has it; the same step on the same contents gives the same
    lens, new, width = [60, 0, 130], [10, 70, 1], 4
    table, free, n_pages = start(lens, width, 5, 3)
    stack, n_free, t = ints(free + [0] * (n_pages - 5)), ints([5]), ints(table)
    out = gb.PagesStep(ints([0] * 4), ints([0] * 3), torch.zeros(81, dtype=torch.int64, device="cuda"), ints([0] * 81), n_free)
    gb.pages_step(ints(lens), ints(new), t, stack, n_free, 81, out=out)
    want = plan(lens, new, table, free, 5, 81, width)
    assert n_free.tolist() == [want[4]] and t.tolist() == want[5] and out.slots.tolist() == want[2]
    n_free.fill_(5)
    gb.pages_step(ints(lens), ints(new), t, stack, n_free, 81, out=out)
    assert n_free.tolist() == [want[4]] and t.tolist() == want[5] and out.slots.tolist() == want[2]


def test_a_request_of_its_rows_whole_length():
    # up to the last token that the table has room for, and a pool of one page
    assert check([0], [64 * 3], 3, 3, 1) == [192]
    assert check([64 * 3 - 1], [1], 3, 0, 1) == [1]
    assert check([0], [64], 1, 1, 1) == [64]
    assert check([0, 0], [1, 1], 1, 1, 1) == [1, 0]
    assert check([0, 5, 0], [65, 1, 1], 4, 1, 1) == [0, 1, 0]       # who needs none is served; who comes after is not


def test_nothing():
    check([5, 0], [0, 0], 2, 1, 1)
    check([5, 0], [0, 0], 2, 1, 1, more=4)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    step = gb.pages_step(e, e, torch.empty(0, 3, dtype=torch.int32, device="cuda"), ints([0, 1]), ints([2]), 2)
    assert step.cu.tolist() == [0] and step.n_free.tolist() == [2] and step.slots.tolist() == [-1, -1]


@pytest.mark.parametrize("lens,keep,new", [(-1, -1, 1), (5, 6, 1), (5, -1, 1), (5, 5, -2), (10, 10, 400), (400, 400, 0),
                                           (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 0, 0), (0, 0, 2 ** 31 - 1)])
def test_numbers_out_of_range_are_left_alone(lens, keep, new):
    # request 1 is not what a request can be: it gets nothing, the others what is theirs
    width, free = 5, [3, 1, 0]
    table = [[8, -7, -7, -7, -7], [4, 5, 6, 2, 9], [7, -7, -7, -7, -7]]
    all_rows = 2 + max(new, 0)
    n_rows = min(all_rows, 2000)
    t, stack = ints(table), ints(free + [0] * 7)
    step = gb.pages_step(ints([64, lens, 63]), ints([1, new, 1]), t, stack, ints([3]), n_rows, keep=ints([64, keep, 63]))
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    table[0][1] = 0
    assert t.tolist() == table and step.n_free.tolist() == [2]
    fits = all_rows <= n_rows      # (rows past the call's: the last request has none of its own either)
    assert step.granted.tolist() == [1, 0, 1 if fits else 0]
    assert step.cu.tolist() == [0, 1, min(1 + max(new, 0), n_rows), min(all_rows, n_rows)]
    slots = step.slots.tolist()
    assert slots[0] == 0 and all(s == -1 for s in slots[1:1 + max(new, 0)])
    if fits:
        assert slots[1 + max(new, 0)] == 7 * 64 + 63


def test_pages_out_of_range_give_no_slot():
    # on the stack and in the table: the tokens that would lie there have no slot
    t, stack = ints([[5, 0], [99, 0]]), ints([1, -3, 2, 0, 0])
    step = gb.pages_step(ints([64, 3]), ints([2, 2]), t, stack, ints([2]), 4)
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert step.slots.tolist() == [-1] * 4 and step.granted.tolist() == [2, 2]
    # a count that is none: nothing is taken
    for count in (-1, 6):
        step = gb.pages_step(ints([64]), ints([1]), ints([[0, 0]]), ints([1, 2, 3, 4, 0]), ints([count]), 1)
        assert gb.check_device_error() == gb.ERR_CACHE_RANGE
        assert step.granted.tolist() == [0] and step.slots.tolist() == [-1] and step.n_free.tolist() == [0]
    # more given back than the pool has
    step = gb.pages_step(ints([128]), ints([0]), ints([[0, 1]]), ints([1, 0, 2]), ints([2]), 0, keep=ints([0]))
    assert gb.check_device_error() == gb.ERR_CACHE_RANGE
    assert step.n_free.tolist() == [3]


@pytest.mark.parametrize("page", [-1, 10, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("B", [2, 300, 1100])
def test_a_page_out_of_range_that_is_given_back_is_reported(B, page):
    # by the step that puts it on the stack, whether it is taken again in it or not; where it stays, nothing is said
    for new, kept in ((0, 64), (1, 64), (0, 65)):
        t, stack = ints([[5, page, 0], [6, 0, 0]] + [[0, 0, 0]] * (B - 2)), ints([1, 2, 3] + [0] * 7)
        lens, keep, more = [100, 3] + [0] * (B - 2), [kept, 3] + [0] * (B - 2), [0, 61 + new] + [0] * (B - 2)
        step = gb.pages_step(ints(lens), ints(more), t, stack, ints([3]), sum(more), keep=ints(keep))
        given_back = kept == 64
        assert gb.check_device_error() == (gb.ERR_CACHE_RANGE if given_back else gb.OK)
        assert stack.tolist()[:4] == ([1, 2, 3, page] if given_back else [1, 2, 3, 0])
        assert step.granted.tolist()[:2] == [0, 61 + new] and step.n_free.tolist() == [3 + given_back - new]
        if new:
            assert t.tolist()[1][1] == page and step.slots.tolist()[-1] == -1


def test_many_steps_keep_every_page_once():
    # a serving run: requests come, grow, are cut back and end; no page is ever two requests' or lost
    r = random.Random(11)
    B, width, n_pages = 24, 12, 150
    lens, table = [0] * B, ints([[-1] * width] * B)
    stack, n_free = ints(list(range(n_pages))), ints([n_pages])
    for step in range(60):
        keep = [0 if r.random() < 0.05 else max(0, x - r.choice([0, 0, 1, 3])) for x in lens]
        new = [r.randint(1, 300) if k == 0 else r.choice([0, 1, 1, 4]) for k in keep]
        new = [min(n, width * PAGE - k) for n, k in zip(new, keep)]
        out = gb.pages_step(ints(lens), ints(new), table, stack, n_free, sum(new), keep=ints(keep))
        granted, n_free = out.granted.tolist(), out.n_free
        lens = [k + g for k, g in zip(keep, granted)]
        rows = table.tolist()
        used = [p for row, x in zip(rows, lens) for p in row[:pages_of(x)]]
        assert sorted(used + stack.tolist()[:int(n_free)]) == list(range(n_pages)), step
        slots = [s for s in out.slots.tolist() if s >= 0]
        assert len(set(slots)) == len(slots) == sum(granted)
