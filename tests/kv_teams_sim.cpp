// Host simulation of how the paged attention shares out its tiles, with the functions that the kernel calls: the choice of
// teams, each team's walk over its segments, the slots that parts of shared segments lie in, and the joins by groups.
// Usage: kv_teams_sim <SMs> <CTAs an SM> <row bytes> <tile> <units> <len> <len> ...
// Checks that every tile is used once, that a warp uses its tiles in the order that it loads them, that every part lies in a slot
// of its own inside the allocation, where the joining team looks for it, and that groups' slots and events are inside theirs.
// Prints the first fault and returns 1, or: tiles, teams, whether they are warps, the most parts of a segment.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <utility>
#include <vector>

#include "../event_driven_persistent_b200/csrc/kv_shared.h"

using namespace et;

#define CHECK(x)                                                          \
    do {                                                                  \
        if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1;        \
    } while (0)

int main(int argc, char** argv) {
    const int n_sm = atoi(argv[1]), grid = n_sm * atoi(argv[2]), row = atoi(argv[3]), tile = atoi(argv[4]), units = atoi(argv[5]);
    const int warps = kKvAttnWarps;
    std::vector<int> pre{0};
    int longest = 0;
    for (int i = 6; i < argc; ++i)
        if (const int n = (atoi(argv[i]) + tile - 1) / tile) {
            pre.push_back(pre.back() + n);
            longest = std::max(longest, n);
        }
    const int live = (int)pre.size() - 1;
    if (live == 0) return printf("0 0 0 0\n"), 0;
    const KvTeams t = kv_choose_teams(pre[live], live, longest, units, grid, warps, kKvShareLog, kKvShareLog, kKvWarpExtra, kv_cta_extra(row), kKvWarpParts);
    CHECK(t.C >= 1 && t.C <= (t.solo ? grid * warps : grid));
    std::vector<char> used((size_t)pre[live] * units);
    std::map<long long, std::pair<int, int>> slots;               // slot -> segment
    std::map<std::pair<int, int>, std::vector<int>> teams_of;     // shared segment -> its teams
    std::map<std::pair<int, int>, std::pair<long long, long long>> numbers;
    std::set<long long> group_slots;
    int most = 1;
    for (int c = 0; c < t.C; ++c) {
        const long long share = kv_share_div(t.N, t.C), t0 = kv_share_begin(c, t.N, t.C, share), t1 = kv_share_begin(c + 1, t.N, t.C, share);
        const int run = (int)(t1 - t0), team = t.solo ? 1 : warps;
        CHECK(run > 0 && run <= kv_longest_run(argc - 6, longest * tile, units, n_sm));
        std::vector<std::vector<std::pair<int, int>>> loads(team), uses(team);  // by warp: (segment's first number, tile counted from t0)
        for (int tw = 0; tw < team; ++tw) {
            KvWalk lw;
            kv_walk_to(lw, pre.data(), live, t.extra, units, t0);
            for (int lt = tw;; lt += team) {
                bool end = false;
                for (;;) {
                    if (lt < lw.s0) lt = lw.s0 + ((tw - lw.s0) & (team - 1));
                    if ((end = lt >= run) || lt < lw.s1) break;
                    kv_walk_next(lw, pre.data(), live, t.extra, units);
                }
                if (end) break;
                loads[tw].push_back({lw.i * units + lw.u, lt - lw.s0});
            }
        }
        std::vector<int> ct(team);
        for (int tw = 0; tw < team; ++tw) ct[tw] = tw;
        KvWalk seg;
        kv_walk_to(seg, pre.data(), live, t.extra, units, t0);
        while (seg.s0 < run) {
            const int s = std::max(seg.s0, 0), e = std::min(seg.s1, run);
            CHECK(s < e && seg.i < live && seg.u < units);
            const std::pair<int, int> at{seg.i, seg.u};
            for (int tw = 0; tw < team; ++tw) {
                if (ct[tw] < s) ct[tw] = s + ((tw - s) & (team - 1));
                for (; ct[tw] < e; ct[tw] += team) {
                    const int k = ct[tw] - seg.s0;
                    CHECK(k >= 0 && k < pre[seg.i + 1] - pre[seg.i]);
                    char& u = used[(size_t)pre[seg.i] * units + (size_t)seg.u * (pre[seg.i + 1] - pre[seg.i]) + k];
                    CHECK(!u);
                    u = 1;
                    uses[tw].push_back({seg.i * units + seg.u, k});
                }
            }
            if (s != seg.s0 || e != seg.s1) {
                const long long slot = (long long)c * kKvMaxSplits + kv_share_slot(c, t0 + seg.s0, t.N, t.C);
                CHECK(slot >= 0 && slot < kv_part_slots(n_sm));
                CHECK(slots.insert({slot, at}).second);
                teams_of[at].push_back(c);
                numbers[at] = {t0 + seg.s0, t0 + seg.s1};
                if (!t.solo) {
                    const long long mine = kv_group_slot(grid, slot);
                    CHECK(mine >= (long long)grid * kKvMaxSplits && mine < kv_part_slots(n_sm) && group_slots.insert(mine).second);
                }
            }
            kv_walk_next(seg, pre.data(), live, t.extra, units);
        }
        for (int tw = 0; tw < team; ++tw) CHECK(loads[tw] == uses[tw]);
    }
    for (char u : used) CHECK(u);
    for (auto& s : teams_of) {
        const auto n = numbers[s.first];
        const KvParts p = kv_parts(n.first, n.second, t.N, t.C);
        CHECK(p.n == (int)s.second.size());
        most = std::max(most, p.n);
        for (int k = 0; k < p.n; ++k) {
            CHECK(s.second[k] == p.c0 + k);
            const auto it = slots.find(kv_part_slot(p, k));
            CHECK(it != slots.end() && it->second == s.first);
        }
        if (p.n > kKvJoin) {
            CHECK(!t.solo && kv_join_groups(p.n) < kv_arrivals(n_sm));  // a team of one warp joins all parts itself
            CHECK((p.n - 1) / kKvJoin < kv_join_groups(p.n));
        }
    }
    printf("%zu %d %d %d\n", used.size(), t.C, (int)t.solo, most);
    return 0;
}
