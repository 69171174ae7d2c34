"""How the tiles of all requests are dealt to teams of warps and the cut heads merged, on the
host: the rules that the kernels take (cache_deal.h), compiled for the CPU and gone through
for whole batches. Each head with tiles has to be finished once, and a merge may read only
parts that were left for it."""
import ctypes
import os
import random
import subprocess

import pytest

from gated_softmax_attention_gb300 import build as gbuild

# The same steps as in the attention kernel (a team finishes the heads that it has whole, leaves a part of
# others, or its block of threads leaves one) and in the merge kernel (the heads that were cut).
SOURCE = r"""
#include <map>
#include <vector>
#include "cache_deal.h"
using namespace gsdpa;

struct Request;
struct Batch {
    using Seq = Request;
    static constexpr bool kJoins = true;
    static constexpr int kSwitch = 1;
    const int* tiles_of;
    int B, Hkv, lg_teams;
};
struct Request {
    int tiles;
    Request(const Batch& a, int b) : tiles(a.tiles_of[b]) {}
    int span() const { return span_of<Batch>(tiles); }
};
struct Head { int b, first, tiles, span; };

enum { FINE = 0, NOT_FINISHED = 1, FINISHED_TWICE = 2, PART_MISSING = 4, PART_OVERWRITTEN = 8, PAST_THE_END = 16 };

// heads_out: how often the first head that is wrong was finished, and which it is
extern "C" int go_through(const int* tiles, int B, int Hkv, int lg, int most_ctas, int* wrong) {
    const Batch a{tiles, B, Hkv, lg};
    const int teams = 1 << lg;
    std::vector<Head> heads;
    std::vector<int> head_at;      // of a place
    for (int b = 0; b < B; ++b)
        for (int h = 0; h < Hkv; ++h) {
            const Request q(a, b);
            for (int k = 0; k < q.span(); ++k) head_at.push_back((int)heads.size());
            heads.push_back({b, (int)head_at.size() - q.span(), q.tiles, q.span()});
        }
    const int N = (int)head_at.size(), ctas = greater(1, lesser(most_ctas, N >> lg));
    const Deal deal(N, ctas << lg);
    int bad = FINE;
    const auto find = [&](int x, int& b, int& rem) {
        b = rem = 0;
        if (x < 0 || x >= N) { bad |= PAST_THE_END; return; }
        const Head& h = heads[head_at[x]];
        b = h.b;
        int at = head_at[x];
        while (at > 0 && heads[at - 1].b == b) --at;
        rem = x - heads[at].first;
    };
    std::vector<int> finished(heads.size());
    std::map<int, int> parts;      // part -> its head
    const auto leave = [&](int part, int head) {
        if (parts.count(part)) bad |= PART_OVERWRITTEN;
        parts[part] = head;
    };
    // ---- the attention kernel
    for (int c = 0; c < ctas; ++c) {
        const JoinedHead joined = joined_head(a, deal, c, find);
        int held = 0;              // teams that have tiles, of a joined head
        for (int k = 0; k < teams; ++k) {
            const int team = (c << lg) + k, from = deal.from(team), to = deal.from(team + 1);
            for (int x = from; x < to;) {
                const Head& h = heads[head_at[x]];
                const int j0 = x - h.first, j1 = lesser(h.tiles, to - h.first);
                if (j1 > j0) {
                    const bool whole = j0 == 0 && j1 == h.tiles && joined.first < 0;
                    if (whole) ++finished[head_at[x]];
                    else if (joined.first >= 0) {
                        if (h.first != joined.first || k != held) bad |= PART_MISSING;
                        ++held;
                    } else leave(part_index(deal, team, h.first), head_at[x]);
                }
                x = h.first + h.span;
            }
        }
        if (joined.first >= 0) {
            if (held != lesser(teams, deal.taker(joined.first + joined.tiles - 1) - (c << lg) + 1)) bad |= PART_MISSING;
            leave(part_index(deal, c << lg, joined.first), head_at[joined.first]);
        }
    }
    // ---- the merge kernel
    const auto merge = [&](int head, int n0, int n1) {
        if (n1 <= n0) return;
        const Head& h = heads[head];
        const Parts<Batch> p(a, deal, n0, n1, h.first, h.span);
        int left = 0;
        for (const auto& x : parts) left += x.second == head;
        if (left != p.n) bad |= PART_MISSING;
        std::map<int, int> seen;
        for (int k = 0; k < p.n; ++k) {
            const int part = part_index(deal, p.team(k), h.first);
            if (!parts.count(part) || parts[part] != head || seen[part]++) bad |= PART_MISSING;
        }
        ++finished[head];
    };
    const int takers = ctas << lg;
    if ((int)heads.size() >= takers) {
        for (int unit = 0; unit < takers - 1; ++unit) {
            const int from = deal.from(unit + 1);
            if (from >= N) continue;
            const Head& h = heads[head_at[from]];
            if (from > h.first && from < h.first + h.tiles && deal.taker(h.first) == unit)
                merge(head_at[from], unit, deal.taker(h.first + h.tiles - 1));
        }
    } else {
        for (int k = 0; k < (int)heads.size(); ++k)
            if (heads[k].tiles > 0) merge(k, deal.taker(heads[k].first), deal.taker(heads[k].first + heads[k].tiles - 1));
    }
    for (int k = (int)heads.size() - 1; k >= 0; --k) {
        const int want = heads[k].tiles > 0;
        if (finished[k] < want) bad |= NOT_FINISHED;
        if (finished[k] > want) bad |= FINISHED_TWICE;
        if (finished[k] != want) *wrong = k;
    }
    return bad;
}
"""


@pytest.fixture(scope="module")
def go_through(tmp_path_factory):
    at = tmp_path_factory.mktemp("deal")
    (at / "deal.cpp").write_text(SOURCE)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + gbuild.CSRC, str(at / "deal.cpp"),
                    "-o", str(at / "deal.so")], check=True)
    lib = ctypes.CDLL(str(at / "deal.so"))

    def call(tiles, H, lg, sms, width=None):
        teams, B = 1 << lg, len(tiles)
        most = min(sms, B * H * -(-(width or max([1, *tiles])) // teams))
        wrong = ctypes.c_int(-1)
        bad = lib.go_through((ctypes.c_int * B)(*tiles), B, H, lg, most, ctypes.byref(wrong))
        return bad, wrong.value
    return call


TEAMS = [0, 1, 2, 3, 4]      # 2^.. teams of a block of threads


@pytest.mark.parametrize("lg", TEAMS)
def test_long_requests_are_finished_once(go_through, lg):
    r = random.Random(lg)
    for _ in range(300):
        B, H = r.randint(1, 12), r.choice([1, 2, 3, 4, 5, 6, 7, 8])
        tiles = [r.choice([0, 40, 64, 200, r.randint(40, 600)]) for _ in range(B)]
        if any(tiles):
            assert go_through(tiles, H, lg, 152) == (0, -1), (tiles, H)


@pytest.mark.parametrize("lg", TEAMS)
@pytest.mark.parametrize("H", [1, 2, 3, 5, 8])
def test_a_head_that_one_team_has_whole(go_through, H, lg):
    # two tiles beside a long request: with two teams the first may have both, and the second only the place after them
    for tiles in ([2, 17], [17, 2], [2, 17, 2], [1, 9], [3, 31]):
        assert go_through(tiles, H, lg, 152) == (0, -1), tiles
    # a single tile among more requests than there are blocks of threads
    for B in (153, 200, 256, 1000):
        for at in (0, 100, B - 1):
            for n in (1, 2, 3):
                tiles = [0] * B
                tiles[at] = n
                assert go_through(tiles, H, lg, 152) == (0, -1), (B, at, n)
    # as many requests of two tiles as there are blocks of threads, and some more
    for B in range(140, 200):
        assert go_through([2] * B, H, lg, 148) == (0, -1), B


@pytest.mark.parametrize("lg", TEAMS)
def test_any_batch_is_finished_once(go_through, lg):
    r = random.Random(100 + lg)
    for _ in range(1000):
        B = r.choice([r.randint(1, 8), r.randint(1, 8), r.randint(9, 200)])
        H = r.randint(1, 8)
        tiles = [r.choice([0, 1, 2, 2, 3, 4, 5, r.randint(1, 40)]) for _ in range(B)]
        if any(tiles):
            assert go_through(tiles, H, lg, r.choice([148, 152])) == (0, -1), (tiles, H)


@pytest.mark.parametrize("lg", TEAMS)
def test_nothing_is_looked_up_where_no_request_has_rows(go_through, lg):
    for B, H in ((1, 1), (64, 8), (200, 1), (8192, 8)):
        assert go_through([0] * B, H, lg, 152, width=4) == (0, -1), (B, H)
