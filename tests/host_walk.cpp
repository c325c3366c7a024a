// Replays on the host how a product's workgroups find their tiles (walk.hpp), for
// offsets as they should be and for offsets that fall, overlap or leave the rows.
// Every tile number must lie among those that launch and workspace are sized for, and
// be given out once; with good offsets every tile is.
#include <walk.hpp>

#include <cstdio>
#include <initializer_list>
#include <random>
#include <vector>

static int g_fail = 0, g_over = 0;

static void replay(const std::vector<int32_t> *offsets, int groups, int64_t rows, int tiles_j, int64_t high, bool tails,
                   bool good) {
    const int32_t *off = offsets ? offsets->data() : nullptr;
    const int most = (int)bakron::row_tiles(high, rows, groups, off != nullptr);
    int slots = 0;  // as the device counts them
    for (int g = 0; g <= groups; ++g) {
        int64_t a, b;
        bakron::rows_of_group(off, groups, rows, g, a, b);
        if (a < 0 || b < a || b > rows) {
            std::fprintf(stderr, "group %d of %d: rows %lld to %lld of %lld\n", g, groups, (long long)a, (long long)b, (long long)rows);
            ++g_fail;
        }
        slots += (int)((b - a + high - 1) / high);
    }
    g_over += slots > most;
    const int64_t launched = (int64_t)most * tiles_j;
    std::vector<int> given(launched, 0);
    for (int tail = 0; tail <= (tails ? 1 : 0); ++tail)
        for (int64_t b = 0; b < (tail ? 128 : launched + 7); ++b) {
            int64_t w;
            int slot, tj;
            if (!bakron::place_of(slots, most, tiles_j, tails, tail, b, w, slot, tj)) continue;
            if (w < 0 || w >= launched || slot < 0 || slot >= slots || tj < 0 || tj >= tiles_j) {
                if (++g_fail < 20)
                    std::fprintf(stderr, "rows %lld groups %d high %lld: workgroup %lld gets tile %lld of %lld\n",
                                 (long long)rows, groups, (long long)high, (long long)b, (long long)w, (long long)launched);
            } else {
                ++given[w];
            }
        }
    const int64_t total = (int64_t)(slots < most ? slots : most) * tiles_j;
    for (int64_t w = 0; w < launched; ++w)
        if (given[w] > 1 || (good && given[w] != (w < total))) ++g_fail;
    if (good && slots > most) ++g_fail;
}

int main() {
    std::mt19937 rng(5);
    auto pick = [&](int64_t n) { return (int64_t)(rng() % (uint64_t)n); };
    for (int64_t rows : {1, 15, 129, 300, 1024, 1500, 9001})
        for (int64_t high : {16, 128, 256})
            for (int tiles_j : {1, 2, 9, 33})
                for (bool tails : {false, true}) {
                    if (tails && high != 256) continue;
                    replay(nullptr, 1, rows, tiles_j, high, tails, true);
                    for (int groups : {1, 3, 5, 8, 63, 64, 200}) {
                        std::vector<int32_t> off(groups + 1);
                        // back and forth over all rows
                        for (int g = 0; g <= groups; ++g) off[g] = g % 2 ? (int32_t)rows : 0;
                        replay(&off, groups, rows, tiles_j, high, tails, false);
                        for (int n = 0; n < 4; ++n) {  // anything at all
                            for (auto &v : off) v = (int32_t)(pick(3 * rows + 2) - rows);
                            replay(&off, groups, rows, tiles_j, high, tails, false);
                        }
                        for (auto &v : off) v = pick(2) ? INT32_MAX : INT32_MIN;
                        replay(&off, groups, rows, tiles_j, high, tails, false);
                        // as they should be, with rows of no group or without
                        for (int n = 0; n < 4; ++n) {
                            int32_t at = 0;
                            for (int g = 0; g <= groups; ++g) {
                                off[g] = at;
                                at += (int32_t)pick((rows - at) / (groups > 8 ? 4 : 2) + 1);
                            }
                            if (n % 2) off[groups] = (int32_t)rows;
                            replay(&off, groups, rows, tiles_j, high, tails, true);
                        }
                    }
                }
    if (g_over == 0) ++g_fail;  // some of the offsets must make more tiles than fit
    if (g_fail) {
        std::fprintf(stderr, "%d failures\n", g_fail);
        return 1;
    }
    std::puts("walk checks passed");
    return 0;
}
