// glr_chain.hpp -- who tells whom what in the recurrence's chain of segments
// (glr.hip): plain index arithmetic, the same for the kernels and on the host.
//
// Segments are counted in processing order.  Segment j publishes its map; the last
// one of a group of G its group's map too; the last one of a block of G groups the
// state that leaves the block.  All of these are words that are set once.
#pragma once

namespace layer {
namespace chain {

constexpr int G = 8;   // segments of a group, groups of a block

constexpr bool closes_group(int j) { return j % G == G - 1; }
constexpr bool closes_block(int j) { return j % (G * G) == G * G - 1; }

// What segment idx reads when the sequence that enters it was itself entered in
// segment src (src = idx: none enters), in the order of time:
//   the block state or the group maps b of `gfirst - far ...`: nb of them, the first
//   one a block state where `far`,
//   the segment maps a of `first ...`: na of them.
struct Reads {
    int first, na, gfirst, nb;
    bool outside, far;   // the sequence was entered before this group; before this block
};
constexpr Reads reads(int idx, int src) {
    const bool entered = src < idx;
    const int g = idx / G, g0 = g * G, first = src > g0 ? src : g0;
    const bool outside = entered && src < g0, far = outside && src / G < g / G * G;
    const int gfirst = far ? g / G * G : src / G;
    return Reads{first, entered ? idx - first : 0, gfirst, outside ? g - gfirst + far : 0, outside, far};
}

// The first segment before idx that still owes one of its words (idx: none).  A
// workgroup that has waited long enough takes this one up: every word of the
// segments before it is there, so it waits for nothing, whether or not its own
// workgroup has started.  The map alone would not do: whoever publishes it may give
// up waiting before the block's state is out, and nobody would take the segment up
// again.  map(j), group(g), state(b): whether the word is there.
template <class Map, class Group, class State>
constexpr int first_unfinished(int idx, Map map, Group group, State state) {
    for (int j = 0; j < idx; j++)
        if (!map(j) || (closes_group(j) && !group(j / G)) || (closes_block(j) && !state(j / (G * G)))) return j;
    return idx;
}

}  // namespace chain
}  // namespace layer
