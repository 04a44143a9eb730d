// How workgroups share a line of units of work in equal parts (awq_tree_attention_prefill.hip): arithmetic
// alone, which a compiler for the CPU takes too.  A line has up to 2^30 units.
#pragma once

#include <cstdint>

namespace awq {

// Units of a share, of so many shares of a line of `all`: enough for all of it, at least `least`, and so many that a
// row tile, of up to `most` units, is in no more than `room` chunks (room 1: borders are kept out of row
// tiles); but no more than there are.
constexpr int share_units(int all, int shares, int least, int most, int room) {
    int each = (int)(((uint32_t)all + (uint32_t)shares - 1) / (uint32_t)shares);
    each = each > least ? each : least;
    const int fewest = room > 1 ? most / (room - 1) + 1 : 1;
    each = each > fewest ? each : fewest;
    return each < all ? each : all > 1 ? all : 1;
}

// The unit that share k begins with.  Shares behind the line's end begin there: with few chunks to a row tile
// that is most of the line (a long sequence among short ones), k times a share's units would pass 32 bits.
constexpr int share_border(int k, int each, int all) {
    const int64_t at = (int64_t)k * each;
    return at < all ? (int)at : all;
}

// The first share that begins at unit `at` (not negative) or behind it, and the last that begins there or before.
constexpr int first_share_from(int at, int each) { return (int)(((uint32_t)at + (uint32_t)each - 1) / (uint32_t)each); }
constexpr int last_share_upto(int at, int each) { return at < 0 ? -1 : (int)((uint32_t)at / (uint32_t)each); }

}  // namespace awq
