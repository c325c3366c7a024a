// walk.hpp -- how the workgroups of a product share its tiles: index arithmetic that
// is the same on the host, which sizes launches and workspaces by it, and the device.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace bakron {

// Group g's rows [a, b), kept inside [0, rows) whatever the offsets hold.  Group
// `groups` stands for the rows after the last group.
__host__ __device__ __forceinline__ void rows_of_group(const int32_t *offsets, int groups, int64_t rows, int g,
                                                       int64_t &a, int64_t &b) {
    if (!offsets) {
        a = g == 0 ? 0 : rows;
        b = rows;
        return;
    }
    auto within = [rows](int64_t v, int64_t low) { return v < low ? low : v > rows ? rows : v; };
    a = g == 0 ? 0 : within(offsets[g], 0);
    b = g == groups ? rows : within(offsets[g + 1], a);
}

// Tiles of `high` rows that `rows` rows in groups make at most: each group, and the
// rows after the last, may end in a partial one.  Launches and workspaces are sized by it.
__host__ __device__ __forceinline__ int64_t row_tiles(int64_t high, int64_t rows, int groups, bool grouped) {
    return (rows + high - 1) / high + (grouped ? groups + 1 : 0);
}

// Workgroups are dealt to the 8 XCDs in turn: XCD x takes the x-th eighth of the
// work, so that tiles that share operands share an L2.
__host__ __device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t total) {
    const int64_t q = total >> 3, r = total & 7, x = b & 7;
    return x * q + (x < r ? x : r) + (b >> 3);
}

// How many of `total` large tiles a launch of them takes.  A last round that would use
// half of the 256 CUs or less is left to small tiles, which, four to a large one, take
// two thirds of a round's time or less (bf16, 16384 rows by 8 groups of
// 11008 x 4096: 1.19 against 1.26 ms; 8192 x 2816 x 4096, 96 tiles left: 162 against
// 166 us).  With more left they do not (8192 x 3328 x 4096, 160 left: 188 against 174).
__host__ __device__ __forceinline__ int64_t without_tail(int64_t total) {
    const int64_t rem = total & 255;
    return total > 256 && rem <= 128 ? total - rem : total;
}

// The place of workgroup b among the tiles of `slots` row tiles by `tiles_j`: its
// number w, row tile and column tile, in bands of 8 row tiles.  has_tail: the launch
// leaves its tail to a launch with `tail`.  `most` is the number of row tiles that launch
// and workspace were sized for: offsets that fall can make groups overlap and `slots`
// larger, and numbers beyond the workspace's tiles must not be given out.  False: no work.
__host__ __device__ __forceinline__ bool place_of(int slots, int most, int tiles_j, bool has_tail, bool tail,
                                                  int64_t b, int64_t &w, int &slot, int &tj) {
    if (slots > most) slots = most;
    const int64_t total = (int64_t)slots * tiles_j, here = has_tail ? without_tail(total) : total;
    if (tail) {
        w = here + b;
        if (w >= total) return false;
    } else {
        if (b >= here) return false;
        w = xcd_order(b, here);
    }
    const int64_t per_band = 8 * (int64_t)tiles_j;
    const int64_t band = w / per_band, in = w - band * per_band;
    const int left = slots - (int)band * 8, width = left < 8 ? left : 8;
    slot = (int)(band * 8) + (int)in % width;
    tj = (int)in / width;
    return true;
}

}  // namespace bakron
