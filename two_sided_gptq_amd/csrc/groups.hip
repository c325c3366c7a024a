// groups.hip -- rows sorted by group and back: bakron_group_sort, bakron_group_gather
// (and _fp8), bakron_group_combine and its gradient.  Groups are a layer's experts, where
// a token has k choices, or the adapters of a batch's requests.
//
// The sort is a stable counting sort.  With c(g) = the number of pairs of groups below g,
// pair i of group g goes to c(g) + the number of pairs of g before i.  Pairs of no group
// are a last group, so order and slots are permutations of all pairs.
//
// Gather, combine and its gradient go by token, not by sorted row: a token's row is read
// once for its k copies (or its k products), and every sorted row is one pair's, so each is
// touched once.  They are bound by HBM.
#include "common.hpp"
#include "elem.hpp"
#include "fp8.hpp"

namespace bakron {
namespace {

constexpr int64_t MAX_PAIRS = int64_t(1) << 24;
constexpr int MAX_GROUPS = 4096;
constexpr int MAX_CHOICES = 64;

// ---------------------------------------------------------------- sort

struct SortArgs {
    const void *ids;
    int wide;  // ids are 64-bit
    int n, groups, bits;
    int32_t *offsets, *order, *slots, *dev_status;
    int32_t *hist;  // [blocks][groups + 1] counts, then their sums over the blocks before
    int32_t *total; // [groups + 1], where scan_kernel ran
    int blocks;
};

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Pair i's group; the last for a negative one and (reported) one that is too large.
// Past the end: one more, which nobody counts.
__device__ __forceinline__ int bin_of(const SortArgs &a, int i, bool &bad) {
    if (i >= a.n) return a.groups + 1;
    const int64_t id = a.wide ? static_cast<const int64_t *>(a.ids)[i] : (int64_t) static_cast<const int32_t *>(a.ids)[i];
    if (id >= a.groups) bad = true;
    return id < 0 || id >= a.groups ? a.groups : (int)id;
}

__device__ __forceinline__ void report(const SortArgs &a, bool bad) {
    if (a.dev_status && __any(bad) && lane_id() == 0) atomicOr(a.dev_status, BAKRON_DEV_BAD_INDEX);
}

// The lanes whose key is this lane's.
__device__ __forceinline__ uint64_t peers_of(int key, int bits) {
    uint32_t lo = ~0u, hi = ~0u;
    for (int b = 0; b < bits; ++b) {
        const int s = key << (31 - b) >> 31;  // all ones where the bit is set
        const uint64_t with = __ballot(s < 0);
        lo &= ~((uint32_t)with ^ s);
        hi &= ~((uint32_t)(with >> 32) ^ s);
    }
    return (uint64_t)hi << 32 | lo;
}

// Adds the wave's 64 keys to count[] and returns how many equal keys the wave had met
// before each.  One lane of each key adds for all of them, in the wave's program order,
// so the result does not depend on the order of atomics.
__device__ __forceinline__ int rank_and_count(int *count, int key, int bits) {
    const uint64_t peers = peers_of(key, bits);
    const int first = __ffsll((unsigned long long)peers) - 1;
    int before = 0;
    if (lane_id() == first) before = atomicAdd(count + key, __popcll(peers));
    before = __shfl(before, first);
    return before + __popcll(peers & ((uint64_t(1) << lane_id()) - 1));
}

// Inclusive sum over the workgroup's threads (WAVES waves); part holds WAVES values.
template <int WAVES>
__device__ __forceinline__ int block_scan(int x, int *part) {
    const int w = threadIdx.x >> 6;
    x = wave_scan(x);
    if (lane_id() == 63) part[w] = x;
    __syncthreads();
    int below = 0;
#pragma unroll
    for (int v = 0; v < WAVES - 1; ++v) below += v < w ? part[v] : 0;
    return x + below;
}

// count[w][b] becomes the first slot of wave w's keys b: base (the pairs of the block
// before, by bin) + smaller bins + earlier waves.  start(b): the bin's first slot.
template <int WAVES, class Total, class Start>
__device__ __forceinline__ void scan_bins(int bins, int *part, Total total, Start start) {
    const int per = (bins + 64 * WAVES - 1) / (64 * WAVES), b0 = threadIdx.x * per;
    int sum = 0;
    for (int b = b0; b < b0 + per && b < bins; ++b) sum += total(b);
    int at = block_scan<WAVES>(sum, part) - sum;
    for (int b = b0; b < b0 + per && b < bins; ++b) {
        const int t = total(b);
        start(b, at);
        at += t;
    }
}

// Few pairs: one workgroup, one launch.  Each wave takes a contiguous stretch.  A wave's ranks
// are a chain of dependent steps, so many waves with few steps each are fastest.
constexpr int ONE_WAVES = 16, ONE_STEPS = 4, ONE_PAIRS = ONE_WAVES * ONE_STEPS * 64, ONE_GROUPS = 1024;

__global__ __launch_bounds__(64 * ONE_WAVES) void sort_one_kernel(SortArgs a) {
    __shared__ int count[ONE_WAVES][ONE_GROUPS + 2];
    __shared__ int part[ONE_WAVES];
    const int lane = lane_id(), w = threadIdx.x >> 6, bins = a.groups + 1;
    const int steps = (a.n + 64 * ONE_WAVES - 1) / (64 * ONE_WAVES);
    int key[ONE_STEPS], rank[ONE_STEPS];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < ONE_STEPS; ++s)
        key[s] = s < steps ? bin_of(a, (w * steps + s) * 64 + lane, bad) : 0;
    for (int b = lane; b <= bins; b += 64) count[w][b] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < ONE_STEPS; ++s)
        if (s < steps) rank[s] = rank_and_count(count[w], key[s], a.bits);
    report(a, bad);
    __syncthreads();
    scan_bins<ONE_WAVES>(
        bins, part,
        [&](int b) {
            int t = 0;
#pragma unroll
            for (int v = 0; v < ONE_WAVES; ++v) t += count[v][b];
            return t;
        },
        [&](int b, int at) {
            a.offsets[b] = at;
            for (int v = 0; v < ONE_WAVES; ++v) {
                const int c = count[v][b];
                count[v][b] = at;
                at += c;
            }
        });
    __syncthreads();
#pragma unroll
    for (int s = 0; s < ONE_STEPS; ++s) {
        const int i = (w * steps + s) * 64 + lane;
        if (s < steps && i < a.n) {
            const int slot = count[w][key[s]] + rank[s];
            a.slots[i] = slot;
            a.order[slot] = i;
        }
    }
}

// Many pairs: blocks of them count their bins; then each block adds up the counts of the
// blocks before it and places its pairs.  From SCAN_BLOCKS blocks on the sums over the
// blocks are a launch of their own.  A block has 8 waves with 4 steps each (65536 pairs, 128
// groups: counting and placing 10.1 us, with 4 waves of 16 steps 16.2), beyond 2^20 pairs
// with 16, which keeps the sums over the blocks short; more than 1024 groups leave LDS for the
// counts of 4 waves only.
constexpr int SCAN_BLOCKS = 64;

template <int WAVES, int STEPS>
__global__ __launch_bounds__(64 * WAVES) void sort_count_kernel(SortArgs a) {
    __shared__ int count[MAX_GROUPS + 2];
    const int bins = a.groups + 1;
    for (int b = threadIdx.x; b <= bins; b += 64 * WAVES) count[b] = 0;
    int key[STEPS];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) key[s] = bin_of(a, (blockIdx.x * STEPS + s) * 64 * WAVES + threadIdx.x, bad);
    report(a, bad);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) atomicAdd(count + key[s], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += 64 * WAVES) a.hist[(int64_t)blockIdx.x * bins + b] = count[b];
}

// A wave a bin.
__global__ __launch_bounds__(256) void sort_scan_kernel(SortArgs a) {
    const int b = blockIdx.x * 4 + (threadIdx.x >> 6), lane = lane_id(), bins = a.groups + 1;
    if (b >= bins) return;
    int sum = 0;
    for (int k0 = 0; k0 < a.blocks; k0 += 64) {
        const int k = k0 + lane;
        int32_t *at = a.hist + (int64_t)k * bins + b;
        const int c = k < a.blocks ? *at : 0;
        const int x = wave_scan(c);
        if (k < a.blocks) *at = sum + x - c;
        sum += __builtin_amdgcn_readlane(x, 63);
    }
    if (lane == 0) a.total[b] = sum;
}

template <int WAVES, int STEPS, bool SCANNED>
__global__ __launch_bounds__(64 * WAVES) void sort_place_kernel(SortArgs a) {
    extern __shared__ int space[];
    const int lane = lane_id(), w = threadIdx.x >> 6, bins = a.groups + 1;
    int *count = space;                                // [WAVES][bins + 1]
    int *total = space + WAVES * (bins + 1);     // [bins]
    int *before = total + bins;                        // [bins]: of this block's bins, in earlier blocks
    int *part = before + bins;
    int key[STEPS], rank[STEPS];
    bool bad = false;
    const int i0 = blockIdx.x * (64 * WAVES * STEPS) + w * STEPS * 64 + lane;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) key[s] = bin_of(a, i0 + s * 64, bad);
    for (int b = threadIdx.x; b < bins; b += 64 * WAVES) {
        if constexpr (SCANNED) {
            total[b] = a.total[b];
            before[b] = a.hist[(int64_t)blockIdx.x * bins + b];
        } else {
            int t = 0, f = 0;
            for (int k0 = 0; k0 < a.blocks; k0 += 32) {
                int c[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) c[k] = k0 + k < a.blocks ? a.hist[(int64_t)(k0 + k) * bins + b] : 0;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    t += c[k];
                    f += k0 + k < (int)blockIdx.x ? c[k] : 0;
                }
            }
            total[b] = t;
            before[b] = f;
        }
    }
    int *mine = count + w * (bins + 1);
    for (int b = lane; b <= bins; b += 64) mine[b] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) rank[s] = rank_and_count(mine, key[s], a.bits);
    __syncthreads();
    scan_bins<WAVES>(
        bins, part, [&](int b) { return total[b]; },
        [&](int b, int at) {
            if (blockIdx.x == 0) a.offsets[b] = at;
            at += before[b];
            for (int v = 0; v < WAVES; ++v) {
                const int c = count[v * (bins + 1) + b];
                count[v * (bins + 1) + b] = at;
                at += c;
            }
        });
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = i0 + s * 64;
        if (i < a.n) {
            const int slot = mine[key[s]] + rank[s];
            a.slots[i] = slot;
            a.order[slot] = i;
        }
    }
}

bool sort_in_one(int64_t n, int groups) { return n <= ONE_PAIRS && groups <= ONE_GROUPS; }
struct SortShape {
    int waves, steps;
    int64_t blocks;
};
SortShape sort_shape(int64_t n, int groups) {
    SortShape y = {groups > ONE_GROUPS ? 4 : 8, 16, 0};
    if (y.waves == 8 && n <= 1 << 20) y.steps = 4;
    y.blocks = (n + 64 * y.waves * y.steps - 1) / (64 * y.waves * y.steps);
    return y;
}

template <int WAVES, int STEPS>
void launch_sort(const SortArgs &a, hipStream_t s) {
    const dim3 grid(a.blocks), block(64 * WAVES);
    const size_t lds = (WAVES * (a.groups + 2) + 2 * (a.groups + 1) + WAVES) * sizeof(int);
    hipLaunchKernelGGL((sort_count_kernel<WAVES, STEPS>), grid, block, 0, s, a);
    if (a.blocks > SCAN_BLOCKS) {
        hipLaunchKernelGGL(sort_scan_kernel, dim3((a.groups + 1 + 3) / 4), dim3(256), 0, s, a);
        hipLaunchKernelGGL((sort_place_kernel<WAVES, STEPS, true>), grid, block, lds, s, a);
    } else {
        hipLaunchKernelGGL((sort_place_kernel<WAVES, STEPS, false>), grid, block, lds, s, a);
    }
}

// ---------------------------------------------------------------- rows

struct RowsArgs {
    const char *x;         // gather: X; combine: Y
    const char *dout;      // gradient of combine
    char *out;             // gather: the sorted rows; combine: the tokens' rows; gradient: dY
    int64_t ldx, ldd, ldo; // in elements
    const int32_t *slots, *end;
    const float *weights;
    float *dweights, *scales;
    int64_t token0;        // the launch's first
    int tokens, k, cols, segs;
    int64_t n;             // pairs
    int past_caches;       // the output goes past the caches
    int32_t *dev_status;
};

// Rows that belong to a group: offsets' last value, kept inside the matrix.
__device__ __forceinline__ int rows_in_groups(const RowsArgs &a) {
    const int e = *a.end;
    return e < 0 ? 0 : e > a.n ? (int)a.n : e;
}

__device__ __forceinline__ int wave_uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A wave takes 512 columns (8 a lane) of a token: the more waves the better, also with many
// tokens (16384 tokens by 4, 4096 columns fp16: 118 us, with two pieces a wave 127, with four 130).
struct Place {
    int64_t token;
    int seg;
};
__device__ __forceinline__ bool place_of_wave(const RowsArgs &a, Place &p) {
    const int64_t wave = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave_uniform(threadIdx.x >> 6);
    const int64_t t = wave / a.segs;
    p.seg = (int)(wave - t * a.segs);
    p.token = a.token0 + t;
    return t < a.tokens;
}

// Lane j holds the slot of the token's j-th choice; -1 for one out of range, and beyond k.
// (k <= 64; slots and weights are passed on with readlane, so every lane has to be active.)
__device__ __forceinline__ int slots_of(const RowsArgs &a, int64_t token) {
    int slot = -1;
    bool bad = false;
    if (lane_id() < a.k) {
        slot = a.slots[token * a.k + lane_id()];
        bad = slot < 0 || slot >= a.n;
    }
    if (a.dev_status && __any(bad) && lane_id() == 0) atomicOr(a.dev_status, BAKRON_DEV_BAD_INDEX);
    return bad ? -1 : slot;
}
__device__ __forceinline__ float weights_of(const RowsArgs &a, int64_t token) {
    return a.weights && lane_id() < a.k ? a.weights[token * a.k + lane_id()] : 1.0f;
}
__device__ __forceinline__ int from_lane(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ float from_lane(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// PIECES x 16 bytes past the caches.  What is written once and is more than the L2s hold
// would only push out what is read: copies of 4096 rows to 16384 of 4096 fp16 in 27.4 instead of
// 33.1 us.
template <int PIECES>
__device__ __forceinline__ void store_past(char *to, const uint32_t *w) {
    typedef uint32_t uintx4 __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
    for (int h = 0; h < PIECES; ++h)
        __builtin_nontemporal_store(uintx4{w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]},
                                    reinterpret_cast<uintx4 *>(to) + h);
}

// Raw elements i .. i + 7; those from `left` on are 0 and not read.
template <int T>
__device__ __forceinline__ void load_raw(const char *base, int64_t i, int left, Raw8<T> &r) {
    constexpr int ES = Raw8<T>::ES;
    if (left >= 8) {
        __builtin_memcpy(r.w, base + i * ES, 8 * ES);
    } else {
#pragma unroll
        for (int q = 0; q < 2 * ES; ++q) r.w[q] = 0;
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) {
                if constexpr (ES == 4)
                    r.w[q] = reinterpret_cast<const uint32_t *>(base)[i + q];
                else
                    r.w[q / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(base)[i + q] << (16 * (q & 1));
            }
    }
}
template <int T>
__device__ __forceinline__ void store_raw(char *base, int64_t i, int left, const Raw8<T> &r, bool past) {
    constexpr int ES = Raw8<T>::ES;
    if (left >= 8) {
        if (past)
            store_past<ES / 2>(base + i * ES, r.w);
        else
            __builtin_memcpy(base + i * ES, r.w, 8 * ES);
    } else {
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) {
                if constexpr (ES == 4)
                    reinterpret_cast<uint32_t *>(base)[i + q] = r.w[q];
                else
                    reinterpret_cast<uint16_t *>(base)[i + q] = (uint16_t)(r.w[q / 2] >> (16 * (q & 1)));
            }
    }
}

// Copies.  fp32 rows go as 16-bit rows of twice the length, so that a lane's 16 bytes lie
// beside its neighbours' (past the caches, two pieces of 16 in every 32 take 1.7 times as long).
__global__ __launch_bounds__(256) void gather_kernel(RowsArgs a) {
    constexpr int T = BAKRON_T_BF16;
    Place p;
    if (!place_of_wave(a, p)) return;
    const int end = rows_in_groups(a), slots = slots_of(a, p.token);
    const int col = p.seg * 512 + lane_id() * 8, left = a.cols - col;
    Raw8<T> r;
    load_raw<T>(a.x, p.token * a.ldx + col, left, r);
    for (int j = 0; j < a.k; ++j) {
        const int slot = from_lane(slots, j);
        if (slot < 0) continue;
        const uint32_t kept = slot < end ? ~0u : 0u;
        Raw8<T> c;
#pragma unroll
        for (int q = 0; q < 4; ++q) c.w[q] = r.w[q] & kept;
        store_raw<T>(a.out, slot * a.ldo + col, left, c, a.past_caches);
    }
}

// Codes past the caches: 65536 rows of 4096 go in 57 instead of 76 us, as the lines that the
// scattered scales fill, 4 bytes at a time, then stay in L2 until they are whole.  (Past
// the caches too, the scales alone take 70 us more.)
__device__ __forceinline__ void store_past(uint8_t *to, uint2 c) {
    typedef uint32_t uintx2 __attribute__((ext_vector_type(2), aligned(1)));
    __builtin_nontemporal_store(uintx2{c.x, c.y}, reinterpret_cast<uintx2 *>(to));
}

// Copies in fp8: 16 lanes hold a block of 128 columns, so its maximum stays inside a
// DPP row; each block is rounded once for all its copies.  A dropped row gets codes 0 and
// scales 1, as a row of zeros would.
template <int T>
__global__ __launch_bounds__(256) void gather_fp8_kernel(RowsArgs a) {
    Place p;
    if (!place_of_wave(a, p)) return;
    const int end = rows_in_groups(a), slots = slots_of(a, p.token);
    const int col = p.seg * 512 + lane_id() * 8, left = a.cols - col;
    float x[8];
    load8<T>(a.x, p.token * a.ldx + col, left, x);
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(x[q]) & 0x7fffffffu);
    m = row_max(m);
    float scale, inv;
    bool bad, used = false;
    block_scale(m, scale, inv, bad);
    const uint2 code = encode8(x, inv, bad);
    uint8_t *out = reinterpret_cast<uint8_t *>(a.out);
    for (int j = 0; j < a.k; ++j) {
        const int slot = from_lane(slots, j);
        if (slot < 0) continue;
        const bool kept = slot < end;
        used |= kept;
        if (left <= 0) continue;
        uint8_t *to = out + slot * a.ldo + col;
        const uint2 c = kept ? code : make_uint2(0, 0);
        if (a.past_caches && left >= 8)
            store_past(to, c);
        else
            store8(to, c, min(8, left));
        if ((lane_id() & 15) == 0) a.scales[(int64_t)(col >> 7) * a.n + slot] = kept ? scale : 1.0f;
    }
    if (bad && used && a.dev_status) atomicOr(a.dev_status, BAKRON_DEV_NONFINITE);
}

constexpr int BATCH = 8;  // rows of a token in flight

// out[t] = sum_j w[t][j] Y[slot[t][j]], in fp32 in the order of j, rounded once.  Dropped
// rows are left out, whatever they hold.
template <int T>
__global__ __launch_bounds__(256) void combine_kernel(RowsArgs a) {
    Place p;
    if (!place_of_wave(a, p)) return;
    const int end = rows_in_groups(a), slots = slots_of(a, p.token);
    const float weights = weights_of(a, p.token);
    const int col = p.seg * 512 + lane_id() * 8, left = a.cols - col;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += BATCH) {
        Raw8<T> r[BATCH];
        int slot[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            slot[j] = j0 + j < a.k ? from_lane(slots, j0 + j) : -1;
            if (slot[j] >= end) slot[j] = -1;
            if (slot[j] >= 0) load_raw<T>(a.x, slot[j] * a.ldx + col, left, r[j]);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (slot[j] >= 0) {
                const float w = from_lane(weights, j0 + j);
                float y[8];
                unpack8<T>(r[j].w, y);
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[q] += w * y[q];
            }
    }
    store8<T>(a.out, p.token * a.ldo + col, left, sum);
}

// Past the caches, 16396 rows of 2050 fp16: 35.2 against 37.7 us; of 4096 bf16 53 against 51.6.  In
// fp32 a lane's two pieces lie 32 bytes from its neighbours', and 10 % more is written than the
// rows hold: 129 against 120 us for 16384 rows of 4096.
template <int T>
__device__ __forceinline__ void store8_past(char *base, int64_t i, const float *x) {
    constexpr int ES = Raw8<T>::ES;
    uint32_t w[2 * ES];
    if constexpr (T == BAKRON_T_F32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(x[q]);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = pack2<T>(x[2 * q], x[2 * q + 1]);
    }
    store_past<ES / 2>(base + i * ES, w);
}

// dY[slot] = w dout[t];  dw[t][j] = <dout[t], Y[slot]>, summed over a lane's columns, the
// lanes and the waves in a fixed order.  WAVES waves take a token.
template <int T, int WAVES, int AT_ONCE>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowsArgs a) {
    __shared__ float part[4][AT_ONCE];
    const int lane = lane_id(), w = wave_uniform(threadIdx.x >> 6), sub = w % WAVES;
    const int64_t at = (int64_t)blockIdx.x * (4 / WAVES) + w / WAVES;
    const bool mine = at < a.tokens;
    const int64_t token = a.token0 + (mine ? at : 0);
    const int end = rows_in_groups(a), slots = slots_of(a, token);
    const float weights = weights_of(a, token);
    const bool past = a.past_caches;
    for (int j0 = 0; j0 < a.k; j0 += AT_ONCE) {
        float dot[AT_ONCE] = {};
        int slot[AT_ONCE];  // -1: none
        float weight[AT_ONCE];
        // here, as lanes leave the loop over columns at different turns
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const bool some = mine && j0 + j < a.k;
            slot[j] = some ? from_lane(slots, j0 + j) : -1;
            weight[j] = some ? from_lane(weights, j0 + j) : 0.0f;
        }
        // what a turn reads is asked for in the turn before
        Raw8<T> d, r[AT_ONCE];
        auto load = [&](int col) {
            const int left = a.cols - col;
            if (left <= 0) return;
            load_raw<T>(a.dout, token * a.ldd + col, left, d);
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j)
                if (slot[j] >= 0 && slot[j] < end) load_raw<T>(a.x, slot[j] * a.ldx + col, left, r[j]);
        };
        int col = (sub * 64 + lane) * 8;
        if (mine) load(col);
        for (; mine && col < a.cols; col += WAVES * 512) {
            const int left = a.cols - col;
            float x[8];
            unpack8<T>(d.w, x);
            Raw8<T> now[AT_ONCE];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) now[j] = r[j];
            load(col + WAVES * 512);
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                if (slot[j] < 0) continue;
                float dy[8] = {};
                if (slot[j] < end) {
                    float y[8];
                    unpack8<T>(now[j].w, y);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        dot[j] += x[q] * y[q];
                        dy[q] = weight[j] * x[q];
                    }
                }
                if (past && left >= 8)
                    store8_past<T>(a.out, slot[j] * a.ldo + col, dy);
                else
                    store8<T>(a.out, slot[j] * a.ldo + col, left, dy);
            }
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            if (j0 + j >= a.k) break;
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        }
        if constexpr (WAVES == 1) {
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j)
                if (mine && lane == 0 && j0 + j < a.k) a.dweights[token * a.k + j0 + j] = dot[j];
        } else {
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j)
                if (lane == 0) part[w][j] = dot[j];
            __syncthreads();
            if (mine && sub == 0 && lane < AT_ONCE && j0 + lane < a.k) {
                float s = 0.0f;
                for (int v = 0; v < WAVES; ++v) s += part[w + v][lane];
                a.dweights[token * a.k + j0 + lane] = s;
            }
            __syncthreads();
        }
    }
}

// A launch stays below 2^32 threads: tokens are taken in several.
template <class Launch>
void by_tokens(RowsArgs a, int64_t tokens, int64_t threads, Launch launch) {
    const int64_t most = (LAUNCH_THREADS - 255) / threads;
    for (int64_t t = 0; t < tokens; t += most) {
        a.token0 = t;
        a.tokens = (int)(tokens - t < most ? tokens - t : most);
        launch(a, dim3((unsigned)((a.tokens * threads + 255) / 256)));
    }
}

// A wave for each 512 columns of a token.
template <class Launch>
void by_pieces(RowsArgs a, int64_t tokens, Launch launch) {
    a.segs = (a.cols + 511) / 512;
    by_tokens(a, tokens, (int64_t)64 * a.segs, launch);
}

template <int T, int WAVES>
void launch_combine_grad(const RowsArgs &a, int64_t tokens, hipStream_t s) {
    by_tokens(a, tokens, 64 * WAVES, [&](const RowsArgs &b, dim3 grid) {
        if (a.k <= 4)
            hipLaunchKernelGGL((combine_grad_kernel<T, WAVES, 4>), grid, dim3(256), 0, s, b);
        else
            hipLaunchKernelGGL((combine_grad_kernel<T, WAVES, BATCH>), grid, dim3(256), 0, s, b);
    });
}

template <int T>
void launch_combine(RowsArgs a, int64_t tokens, hipStream_t s) {
    if (!a.dout) {
        by_pieces(a, tokens,
                  [&](const RowsArgs &b, dim3 grid) { hipLaunchKernelGGL(combine_kernel<T>, grid, dim3(256), 0, s, b); });
    } else if (a.cols <= 512) {
        launch_combine_grad<T, 1>(a, tokens, s);
    } else if (a.cols <= 1024) {
        launch_combine_grad<T, 2>(a, tokens, s);
    } else {  // 16384 rows of 4096 bf16 in 53 us, 16396 of 2050 fp16 in 35
        launch_combine_grad<T, 4>(a, tokens, s);
    }
}

template <class F>
void by_type(int32_t type, F f) {
    if (type == BAKRON_T_F32)
        f(std::integral_constant<int, BAKRON_T_F32>());
    else if (type == BAKRON_T_BF16)
        f(std::integral_constant<int, BAKRON_T_BF16>());
    else
        f(std::integral_constant<int, BAKRON_T_F16>());
}

bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// With fewer bytes than the L2s hold, whoever comes next finds them there.
bool many(int64_t bytes) { return bytes > int64_t(32) << 20; }

int32_t check_rows(int32_t type, int64_t tokens, int32_t k, int64_t cols, int32_t groups) {
    BK_REQUIRE(type == BAKRON_T_F32 || type == BAKRON_T_BF16 || type == BAKRON_T_F16, "bad type %d", type);
    BK_REQUIRE(tokens >= 1 && k >= 1 && k <= MAX_CHOICES && tokens <= MAX_PAIRS / k && cols >= 1 && cols <= MAX_PAIRS,
               "bad sizes tokens=%lld k=%d cols=%lld", (long long)tokens, k, (long long)cols);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    return BAKRON_OK;
}

int32_t check_stride(const char *name, int64_t ld, int64_t cols) {
    BK_REQUIRE(ld >= cols && ld <= MAX_LD, "bad row stride %s=%lld for %lld columns", name, (long long)ld,
               (long long)cols);
    return BAKRON_OK;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

#define BK_TRY(expr)                          \
    do {                                      \
        int32_t bk_r_ = (expr);               \
        if (bk_r_ != BAKRON_OK) return bk_r_; \
    } while (0)

extern "C" size_t bakron_group_sort_workspace_size(int64_t n, int32_t groups) {
    if (n < 1 || n > MAX_PAIRS || groups < 1 || groups > MAX_GROUPS || sort_in_one(n, groups)) return 0;
    return align256(sort_shape(n, groups).blocks * (groups + 1) * sizeof(int32_t)) + align256((groups + 1) * sizeof(int32_t));
}

extern "C" int32_t bakron_group_sort(const void *ids, int32_t id_bits, int64_t n, int32_t groups, int32_t *offsets,
                                     int32_t *order, int32_t *slots, int32_t *dev_status, void *ws, size_t ws_bytes,
                                     void *stream_) {
    clear_error();
    BK_REQUIRE(ids && offsets && order && slots, "ids, offsets, order and slots must be non-NULL");
    BK_REQUIRE(id_bits == 32 || id_bits == 64, "id_bits must be 32 or 64, not %d", id_bits);
    BK_REQUIRE(n >= 1 && n <= MAX_PAIRS, "bad size n=%lld", (long long)n);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    BK_REQUIRE(aligned(ids, id_bits / 8), "ids are misaligned for their type");
    const size_t need = bakron_group_sort_workspace_size(n, groups);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) {
        set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, ws_bytes);
        return BAKRON_ERR_WORKSPACE;
    }
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    SortArgs a = {};
    a.ids = ids, a.wide = id_bits == 64, a.n = (int)n, a.groups = groups;
    while ((groups + 1) >> a.bits) ++a.bits;
    a.offsets = offsets, a.order = order, a.slots = slots, a.dev_status = dev_status;
    if (sort_in_one(n, groups)) {
        hipLaunchKernelGGL(sort_one_kernel, dim3(1), dim3(64 * ONE_WAVES), 0, s, a);
        BK_LAUNCH_CHECK("sort_one_kernel");
        return BAKRON_OK;
    }
    const SortShape y = sort_shape(n, groups);
    a.blocks = (int)y.blocks;
    Carver c(ws);
    a.hist = c.take<int32_t>((size_t)a.blocks * (groups + 1));
    a.total = c.take<int32_t>(groups + 1);
    if (y.waves == 4)
        launch_sort<4, 16>(a, s);
    else if (y.steps == 4)
        launch_sort<8, 4>(a, s);
    else
        launch_sort<8, 16>(a, s);
    BK_LAUNCH_CHECK("group sort");
    return BAKRON_OK;
}

extern "C" int32_t bakron_group_gather(const void *X, int32_t type, int64_t tokens, int32_t k, int64_t cols, int64_t ldx,
                                       const int32_t *slots, int32_t groups, const int32_t *offsets, void *out,
                                       int64_t ldo, int32_t *dev_status, void *stream_) {
    clear_error();
    BK_REQUIRE(X && slots && offsets && out, "X, slots, offsets and out must be non-NULL");
    BK_TRY(check_rows(type, tokens, k, cols, groups));
    BK_TRY(check_stride("ldx", ldx, cols));
    BK_TRY(check_stride("ldo", ldo, cols));
    BK_REQUIRE(aligned(X, elem_size(type)) && aligned(out, elem_size(type)), "X or out is misaligned for its type");
    BK_TRY(check_device());
    RowsArgs a = {};
    a.x = static_cast<const char *>(X), a.out = static_cast<char *>(out), a.ldx = ldx, a.ldo = ldo;
    a.slots = slots, a.end = offsets + groups, a.k = k, a.cols = (int)cols, a.n = tokens * k, a.dev_status = dev_status;
    // rows off 16 bytes leave parts of lines (16384 rows of 2050 fp16: 18.5 past the caches, 15.6 else)
    a.past_caches = many(a.n * cols * elem_size(type)) && ldo * elem_size(type) % 16 == 0 && aligned(out, 16);
    if (type == BAKRON_T_F32) a.cols *= 2, a.ldx *= 2, a.ldo *= 2;
    by_pieces(a, tokens, [&](const RowsArgs &b, dim3 grid) {
        hipLaunchKernelGGL(gather_kernel, grid, dim3(256), 0, static_cast<hipStream_t>(stream_), b);
    });
    BK_LAUNCH_CHECK("gather_kernel");
    return BAKRON_OK;
}

extern "C" int32_t bakron_group_gather_fp8(const void *X, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                                           int64_t ldx, const int32_t *slots, int32_t groups, const int32_t *offsets,
                                           uint8_t *Q, int64_t ldq, float *scales, int32_t *dev_status, void *stream_) {
    clear_error();
    BK_REQUIRE(X && slots && offsets && Q && scales, "X, slots, offsets, Q and scales must be non-NULL");
    BK_TRY(check_rows(type, tokens, k, cols, groups));
    BK_TRY(check_stride("ldx", ldx, cols));
    BK_TRY(check_stride("ldq", ldq, cols));
    BK_REQUIRE(aligned(X, elem_size(type)), "X is misaligned for its type");
    BK_TRY(check_device());
    RowsArgs a = {};
    a.x = static_cast<const char *>(X), a.out = reinterpret_cast<char *>(Q), a.ldx = ldx, a.ldo = ldq;
    a.slots = slots, a.end = offsets + groups, a.k = k, a.cols = (int)cols, a.n = tokens * k, a.scales = scales;
    a.past_caches = many(a.n * cols);
    a.dev_status = dev_status;
    by_type(type, [&](auto t) {
        by_pieces(a, tokens, [&](const RowsArgs &b, dim3 grid) {
            hipLaunchKernelGGL(gather_fp8_kernel<t.value>, grid, dim3(256), 0, static_cast<hipStream_t>(stream_), b);
        });
    });
    BK_LAUNCH_CHECK("gather_fp8_kernel");
    return BAKRON_OK;
}

extern "C" int32_t bakron_group_combine(const void *Y, int32_t type, int64_t tokens, int32_t k, int64_t cols,
                                        int64_t ldy, const int32_t *slots, int32_t groups, const int32_t *offsets,
                                        const float *weights, void *out, int64_t ldo, int32_t *dev_status,
                                        void *stream_) {
    clear_error();
    BK_REQUIRE(Y && slots && offsets && out, "Y, slots, offsets and out must be non-NULL");
    BK_TRY(check_rows(type, tokens, k, cols, groups));
    BK_TRY(check_stride("ldy", ldy, cols));
    BK_TRY(check_stride("ldo", ldo, cols));
    BK_REQUIRE(aligned(Y, elem_size(type)) && aligned(out, elem_size(type)), "Y or out is misaligned for its type");
    BK_TRY(check_device());
    RowsArgs a = {};
    a.x = static_cast<const char *>(Y), a.out = static_cast<char *>(out), a.ldx = ldy, a.ldo = ldo;
    a.slots = slots, a.end = offsets + groups, a.weights = weights, a.k = k, a.cols = (int)cols, a.n = tokens * k;
    a.dev_status = dev_status;
    by_type(type, [&](auto t) { launch_combine<t.value>(a, tokens, static_cast<hipStream_t>(stream_)); });
    BK_LAUNCH_CHECK("combine_kernel");
    return BAKRON_OK;
}

extern "C" int32_t bakron_group_combine_grad(const void *dout, int64_t ldd, const void *Y, int32_t type, int64_t tokens,
                                             int32_t k, int64_t cols, int64_t ldy, const int32_t *slots, int32_t groups,
                                             const int32_t *offsets, const float *weights, void *dY, int64_t lddy,
                                             float *dweights, int32_t *dev_status, void *stream_) {
    clear_error();
    BK_REQUIRE(dout && Y && slots && offsets && weights && dY && dweights,
               "dout, Y, slots, offsets, weights, dY and dweights must be non-NULL");
    BK_TRY(check_rows(type, tokens, k, cols, groups));
    BK_TRY(check_stride("ldd", ldd, cols));
    BK_TRY(check_stride("ldy", ldy, cols));
    BK_TRY(check_stride("lddy", lddy, cols));
    BK_REQUIRE(aligned(dout, elem_size(type)) && aligned(Y, elem_size(type)) && aligned(dY, elem_size(type)),
               "dout, Y or dY is misaligned for its type");
    BK_TRY(check_device());
    RowsArgs a = {};
    a.x = static_cast<const char *>(Y), a.dout = static_cast<const char *>(dout), a.out = static_cast<char *>(dY);
    a.ldx = ldy, a.ldd = ldd, a.ldo = lddy, a.slots = slots, a.end = offsets + groups, a.weights = weights;
    a.dweights = dweights, a.k = k, a.cols = (int)cols, a.n = tokens * k, a.dev_status = dev_status;
    a.past_caches = many(a.n * cols * elem_size(type));
    by_type(type, [&](auto t) { launch_combine<t.value>(a, tokens, static_cast<hipStream_t>(stream_)); });
    BK_LAUNCH_CHECK("combine_grad_kernel");
    return BAKRON_OK;
}
