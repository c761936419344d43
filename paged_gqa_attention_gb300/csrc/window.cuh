// window.cuh -- which tokens a sliding window with visible first tokens shows, and the list of
// tiles that hold them, for the kernels that walk it.
#pragma once

#include "common.cuh"

namespace pa {

// The tokens that queries first .. last of a sequence may see under window and sinks are
// [0, s) and [lo, last]: lo = max(0, first - window + 1), s = the sinks before it (0 when the
// sinks reach the window: then the whole range from lo = 0 is visible).
// Tiles of kTile tokens that hold one are numbered in order: tile v < n_sink is context tile v,
// later ones are context tiles from w0 on.  (A tile holding both the last sink and the
// window's first token counts once, among the sinks.)
template <int kTile>
struct WindowTiles {
    int s, lo;
    int n_sink, w0, n;

    __device__ __forceinline__ WindowTiles(int window, int sinks, int first, int last) {
        lo = max(0, first - window + 1);
        s = sinks;
        if (s >= lo) s = lo = 0;
        n_sink = (s + kTile - 1) / kTile;
        w0 = max(lo / kTile, n_sink);
        n = n_sink + max(0, last / kTile + 1 - w0);
    }
    // context tile of list entry v
    __device__ __forceinline__ int tile(int v) const { return v < n_sink ? v : w0 + (v - n_sink); }
    // whether position p (not past the last query) is seen by the first query
    __device__ __forceinline__ bool sees(int p) const { return p < s || p >= lo; }
    // whether any position of [p, p + len) is, for len at most a tile
    __device__ __forceinline__ bool sees_any(int p, int len) const { return p < s || p + len > lo; }
};

// The same tokens as one list of rows: the sinks, rounded up to groups of 16, then the window from
// the group of 16 that holds its first token on.
struct WindowRows {
    int s, lo;      // as above; rows in between (at the ends of the groups) are seen by no query
    int s16;        // rows of the sinks (0 when the list is one range from position 0)
    int shift;      // row r >= s16 is position r + shift
    int rows;       // up to the last query's own position

    __device__ __forceinline__ void set(int window, int sinks, int first, int last) {
        lo = max(0, first - window + 1);
        s = sinks;
        if (s >= lo) s = lo = 0;
        s16 = (s + 15) & ~15;
        const int lo16 = lo & ~15;
        if (s16 >= lo16) s16 = shift = 0;   // nothing to leave out
        else shift = lo16 - s16;
        rows = last + 1 - shift;
    }
    __device__ __forceinline__ int position(int r) const { return r < s16 ? r : r + shift; }
};

}  // namespace pa
