// A model of how the recurrence's workgroups wait for one another (csrc/glr.hip), on
// the host and with the kernel's own rules (csrc/glr_chain.hpp): which words a segment
// reads, and which segment a workgroup takes up after it has waited long enough.
// Workgroups start in any order into a limited number of slots, which they keep until
// their own segment is done, and take their steps in any order.
#include <random>
#include <vector>

#include "../chunked_gated_delta_08_amd/csrc/glr_chain.hpp"

namespace {

using namespace layer::chain;

struct Words {
    std::vector<char> map, group, state;
};

enum Phase { TELL_MAP, TELL_GROUP, READ, DONE };
struct Group {   // a workgroup
    int own, seg, tries = 0;
    Phase phase = TELL_MAP;
};

struct Model {
    int nseg, polls;
    bool maps_only;              // the rule without the groups' and blocks' words
    std::vector<int> src;        // per segment: where the sequence that enters it was entered
    Words w;

    bool maps_there(const Reads& r) const {
        for (int i = 0; i < r.na; i++)
            if (!w.map[r.first + i]) return false;
        return true;
    }
    bool groups_there(int j, const Reads& r) const {
        for (int i = 0; i < r.nb; i++)
            if (!(r.far && i == 0 ? w.state[j / G / G - 1] : w.group[r.gfirst + i - r.far])) return false;
        return true;
    }
    // One step; false once the workgroup has ended.
    bool step(Group& g) {
        const int j = g.seg;
        const Reads r = reads(j, src[j]);
        const bool later = j + 1 < nseg, closes = later && closes_group(j);
        bool there = true;
        switch (g.phase) {
            case TELL_MAP:
                if (later) w.map[j] = 1;
                g.phase = closes ? TELL_GROUP : READ;
                return true;
            case TELL_GROUP:
                there = maps_there(r);
                if (there) w.group[j / G] = 1, g.phase = READ, g.tries = 0;
                break;
            case READ:
                there = src[j] == j || ((closes || maps_there(r)) && groups_there(j, r));
                if (there) g.phase = DONE, g.tries = 0;
                break;
            case DONE:
                if (later && closes_block(j)) w.state[j / G / G] = 1;
                if (j == g.own) return false;
                g.seg = g.own, g.phase = TELL_MAP;
                return true;
        }
        if (there || ++g.tries < polls) return true;
        g.tries = 0, g.phase = TELL_MAP;
        const auto yes = [](int) { return true; };
        const auto map = [&](int i) { return w.map[i] != 0; };
        if (maps_only) g.seg = first_unfinished(g.own, map, yes, yes);
        else
            g.seg = first_unfinished(g.own, map, [&](int i) { return w.group[i] != 0; },
                                     [&](int i) { return w.state[i] != 0; });
        return true;
    }
};

}  // namespace

// Whether all workgroups end.  `order`: the segments in which they start; `begins`:
// segments inside which a sequence begins (the first one begins in segment 0).
extern "C" int glr_chain_ends(int nseg, const int* order, int slots, int polls, int maps_only, const int* begins,
                              int nbegins, unsigned seed) {
    std::mt19937 rng(seed);
    Model m{nseg, polls, maps_only != 0, std::vector<int>(nseg), {}};
    m.w = Words{std::vector<char>(nseg), std::vector<char>(nseg), std::vector<char>(nseg)};
    for (int j = 0, b = -1; j < nseg; j++) {
        m.src[j] = b < 0 ? 0 : begins[b];
        while (b + 1 < nbegins && begins[b + 1] == j) b++;
    }
    std::vector<Group> in;
    int next = 0;
    // Some workgroups are slow: they take one step where others take a hundred.
    std::vector<char> slow(nseg);
    for (auto& s : slow) s = rng() % 4 == 0;
    long idle = 0;
    while (next < nseg || !in.empty()) {
        while ((int)in.size() < slots && next < nseg) in.push_back(Group{order[next], order[next]}), next++;
        const size_t i = rng() % in.size();
        if (slow[in[i].own] && rng() % 100 != 0) continue;
        const Words before = m.w;
        const bool more = m.step(in[i]);
        if (!more) in[i] = in.back(), in.pop_back();
        idle = more && before.map == m.w.map && before.group == m.w.group && before.state == m.w.state ? idle + 1 : 0;
        // Between two changes each of the `slots` workgroups has every step of a pass through
        // two segments (at most 4 + 2 polls each) many times over, the slow ones too.
        if (idle > 2000l * slots * (8 + 4 * polls)) return 0;
    }
    return 1;
}

// Whether reads(idx, src) names each thing that enters idx once: from src on to idx,
// every segment in one map, one group's map or the block's state.
extern "C" int glr_chain_reads_cover(int nseg) {
    for (int idx = 0; idx < nseg; idx++)
        for (int src = 0; src <= idx; src++) {
            const Reads r = reads(idx, src);
            if (src == idx) {
                if (r.na || r.nb || r.outside || r.far) return 0;
                continue;
            }
            if (r.na > G - 1 || r.nb > G) return 0;
            int at = src;   // the next segment to be accounted for
            for (int i = 0; i < r.nb; i++) {
                if (r.far && i == 0) {
                    const int b = idx / G / G - 1;
                    if (src > b * G * G + G * G - 1) return 0;
                    at = (b + 1) * G * G;
                } else {
                    const int g = r.gfirst + i - r.far;
                    if (at < g * G || at >= (g + 1) * G) return 0;
                    at = (g + 1) * G;
                }
            }
            for (int i = 0; i < r.na; i++)
                if (r.first + i != at++) return 0;
            if (at != idx) return 0;
        }
    return 1;
}
