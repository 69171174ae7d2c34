// cache_deal.h -- how the tiles of all sequences and K/V heads are dealt to teams of
// warps, and who leaves and who merges the parts of a head that several teams share.
// Whole numbers only, which the host tests go through as the kernels do. Not part of
// the public ABI.
//
// A kernel's arguments A have the members used here and
//   A::Seq(a, b)   sequence b: tiles, span()
//   lg_teams       teams of a CTA, 2^lg_teams
//   kJoins         a CTA whose share is all of one head leaves one part
//   kSwitch        most places after a head without a tile
#pragma once

#ifdef __CUDACC__
#define GSDPA_DEAL __device__ __forceinline__
#else
#define GSDPA_DEAL inline
#endif

namespace gsdpa {

GSDPA_DEAL int lesser(int a, int b) { return a < b ? a : b; }
GSDPA_DEAL int greater(int a, int b) { return a > b ? a : b; }

// Places of a head in the sequence of all tiles: after its tiles come some without
// one. A team that goes on to another head stores what it has, reads other
// queries and has, at a sequence's end, an open block of twice the bytes, which
// even shares of the tiles alone do not show: of 1216 teams with 11 tiles each of
// 24 sequences of up to 32767 tokens, the 48 that went on ended 5 us after the
// others. (Measured, 8 bits, with 2, 4, 6 and 8 places: that 52.2, 50.4, 50.9, 51.5 us, up
// to 5000 tokens 19.3, 17.7, 17.5, 17.9; 64 x 200 tokens, heads of 4 tiles, 18.4,
// 21.0, 20.3, 20.1. 4 bits, where a team is one warp that ends a head without a barrier and
// takes longer for a tile, with 0, 1, 2, 4 and 6: 200 sequences of up to 1500 tokens 69.6, 66.5, 69.6,
// 72.1, 71.3 us; 24 of up to 32767 47.8, 46.5, 46.8, 46.5, 47.2; 64 x 8192 with the gate 132.1, 134, 134.5,
// 134, 138; 7 of up to 4099, 5 rows, 16.7, 16.5, 16.4, 16.1, 16.1.)
template <class A>
GSDPA_DEAL int span_of(int tiles) {
    return tiles + lesser(A::kSwitch, tiles / 2);
}

// n things dealt to k takers in order, each as many as the next or one more:
// where a taker's share begins, and whose share holds thing x.
struct Deal {
    int each, more;
    GSDPA_DEAL Deal(int n, int k) : each(n / k), more(n % k) {}
    GSDPA_DEAL int from(int c) const { return c * each + lesser(c, more); }
    GSDPA_DEAL int taker(int x) const {
        const int fat = more * (each + 1);
        return x < fat ? x / (each + 1) : more + (x - fat) / each;
    }
};

// Which part team n leaves of the cut head whose first tile is u0: of the first
// head of its share, or of the last.
GSDPA_DEAL int part_index(const Deal& deal, int n, int u0) { return 2 * n + (u0 <= deal.from(n) ? 0 : 1); }

// Whether the places [from, to) of a CTA, the first of them a tile, are all of the cut head
// at [u0, u0 + span): its teams' parts are then joined and left as one, its first team's. (Asked of cut
// heads only. One that a team has whole that team finishes, and the merge does not look at it, though
// the CTA's other teams may have nothing but the head's last place, which is no tile, or nothing at all.)
GSDPA_DEAL bool joins(int lg_teams, int from, int to, int u0, int span) {
    return lg_teams > 0 && from >= u0 && to <= u0 + span;
}

// The head whose parts the teams of CTA c join: its first place and its tiles; first -1 where
// they do not. find(x, b, rem): place x is place rem of sequence b.
struct JoinedHead {
    int first, tiles;
};
template <class A, class Find>
GSDPA_DEAL JoinedHead joined_head(const A& a, const Deal& deal, int c, Find find) {
    const int from = deal.from(c << a.lg_teams), to = deal.from((c + 1) << a.lg_teams);
    if (from >= to) return {-1, 0};   // (no tile at all: place 0 is no request's)
    int b, rem;
    find(from, b, rem);
    const typename A::Seq q(a, b);
    const int first = from - rem % greater(q.span(), 1);
    // (cut: tiles before the CTA's share, or more of them than its first team has)
    const bool cut = first < from || q.tiles > deal.from((c << a.lg_teams) + 1) - from;
    if (cut && from < first + q.tiles && joins(a.lg_teams, from, to, first, q.span())) return {first, q.tiles};
    return {-1, 0};
}

// The parts of a cut head that teams first .. last have tiles of: one each, or one of a
// CTA whose teams' are joined (any CTA but those of the first and the last team, and maybe these).
template <class A>
struct Parts {
    int n;             // how many
    int n0, lead, mid, lg;   // first team; parts of its CTA; CTAs between that and the last team's
    GSDPA_DEAL Parts(const A& a, const Deal& deal, int first, int last, int u0, int span) : n0(first) {
        n = last - first + 1;
        if constexpr (A::kJoins) {
            lg = a.lg_teams;
            const int c0 = first >> lg, c1 = last >> lg;
            const auto joined = [&](int c) { return joins(lg, deal.from(c << lg), deal.from((c + 1) << lg), u0, span); };
            lead = joined(c0) ? 1 : lesser(last, ((c0 + 1) << lg) - 1) - first + 1;
            mid = greater(c1 - c0 - 1, 0);
            n = lead + mid + (c1 == c0 ? 0 : (joined(c1) ? 1 : last - (c1 << lg) + 1));
        }
    }
    GSDPA_DEAL int team(int k) const {
        if constexpr (A::kJoins) {
            const int c0 = n0 >> lg;
            if (k >= lead) return k < lead + mid ? (c0 + 1 + k - lead) << lg : ((c0 + 1 + mid) << lg) + (k - lead - mid);
        }
        return n0 + k;
    }
};

}  // namespace gsdpa
