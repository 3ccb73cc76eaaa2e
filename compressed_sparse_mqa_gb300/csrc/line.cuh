// line.cuh -- one line of work over a list of entries (sessions, groups of sessions), walked by a
// warp, 32 entries at a time: entry i has units_of(i) >= 0 units, and they follow one another.
// Every CTA walks the same line and takes its own share of it, so no kernel has to lay it out first.
#pragma once

#include "ds4a_common.cuh"

namespace ds4a {

struct Line {
    int first;                       // first entry of the group of 32
    long long before, mine, incl;    // units before the group; this lane's entry's; up to and with it
};

template <typename F>
DS4A_DEVINL void line_load(Line &k, int n, int first, long long before, F units_of) {
    const int lane = threadIdx.x & 31;
    k.first = first;
    k.before = before;
    k.mine = first + lane < n ? units_of(first + lane) : 0;
    k.incl = k.mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, k.incl, o);
        if (lane >= o) k.incl += up;
    }
}
DS4A_DEVINL long long line_end(const Line &k) { return k.before + __shfl_sync(0xffffffffu, k.incl, 31); }

// Moves to the group of unit u (not before the present one's); the lane whose entry has it, or -1 behind the last.
template <typename F>
DS4A_DEVINL int line_to(Line &k, int n, long long u, F units_of) {
    for (;;) {
        const long long end = line_end(k);
        if (u < end) return __ffs(__ballot_sync(0xffffffffu, k.before + k.incl > u)) - 1;
        if (k.first + 32 >= n) return -1;
        line_load(k, n, k.first + 32, end, units_of);
    }
}

// Units of the whole line; the walk is at its first group behind it.
template <typename F>
DS4A_DEVINL long long line_total(Line &k, int n, F units_of) {
    line_load(k, n, 0, 0, units_of);
    if (n <= 32) return line_end(k);
    while (k.first + 32 < n) line_load(k, n, k.first + 32, line_end(k), units_of);
    const long long total = line_end(k);
    line_load(k, n, 0, 0, units_of);
    return total;
}

// non-negative a / b; in 32 bits when they fit, as they do but for lines of millions of tiles
DS4A_DEVINL long long line_quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b)) : a / b;
}

}  // namespace ds4a
