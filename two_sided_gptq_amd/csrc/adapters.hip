// adapters.hip -- low-rank adapters of many requests beside a shared projection:
// bakron_adapter_matmul and its gradients.
//
// Row r of group (adapter) g:  out[r] = base[r] + s_g B_g (A_g x_r), A_g rank x K, B_g N x rank.
//   P = s X A^T,  out = base + P B^T
//   U = s dY B,   dX = base + U A,  dA_g = U_g^T X_g,  dB_g = dY_g^T P_g
// All rows of a group share its matrices; `order` names the rows of each place, so that
// neither X nor the output has to be sorted.  The rank is small: every product is bound by
// the bytes of X, dY and the outputs, and the matrix cores have time to spare.
//
// shrink_kernel makes P (or U): a workgroup takes a tile of 16 MT places of one group, its
// waves share K.  expand_kernel adds P B^T to the base, a wave 64 columns at a time.
// outer_kernel sums over a group's places.  In between P and U are kept as two bf16 numbers
// each, x = hi + lo (2^-16 |x| is lost): the products with both parts are exact in
// fp32 sums, and neither fp16's range nor bf16's 8 bits limit what lies between two products.
#include <algorithm>

#include "common.hpp"
#include "elem.hpp"
#include "walk.hpp"

namespace bakron {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int64_t MAX_DIM = int64_t(1) << 24;
constexpr int MAX_GROUPS = 4096;
constexpr int MAX_RANK = 256;

template <int T>
__device__ __forceinline__ floatx4 mfma(uintx4 a, uintx4 b, floatx4 c) {
    if constexpr (T == BAKRON_T_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
}
__device__ __forceinline__ floatx4 mfma_bf16(uintx4 a, uintx4 b, floatx4 c) { return mfma<BAKRON_T_BF16>(a, b, c); }

// 8 values of a 16-bit type; those from `left` on are 0 and not read.
__device__ __forceinline__ uintx4 load_frag(const char *base, int64_t i, int left) {
    uintx4 r = {0, 0, 0, 0};
    if (left >= 8) {
        __builtin_memcpy(&r, base + 2 * i, 16);
    } else {
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < left) r[q / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(base)[i + q] << (16 * (q & 1));
    }
    return r;
}
__device__ __forceinline__ uintx4 load_whole(const char *base, int64_t i) {
    uintx4 r;
    __builtin_memcpy(&r, base + 2 * i, 16);
    return r;
}

// x as two bf16 numbers, hi in the upper half.
__device__ __forceinline__ uint32_t pack_parts(float x) {
    const uint32_t hi = f32_to_bf16(x);
    const float h = __uint_as_float(hi << 16);
    const uint32_t lo = __builtin_isfinite(h) ? f32_to_bf16(x - h) : 0;
    return hi << 16 | lo;
}
// 8 packed numbers as the two operands' fragments.
__device__ __forceinline__ void unpack_parts(const uint32_t *x, uintx4 &hi, uintx4 &lo) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302);
        lo[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100);
    }
}
// 8 fp16 values as bf16 parts, exactly: 11 bits are 8 and what is left.
__device__ __forceinline__ void split_f16(uintx4 v, uintx4 &hi, uintx4 &lo) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = f16_to_f32((uint16_t)v[j]), b = f16_to_f32((uint16_t)(v[j] >> 16));
        const uint32_t ah = __float_as_uint(a), bh = __float_as_uint(b);
        hi[j] = __builtin_amdgcn_perm(bh, ah, 0x07060302);
        const float al = a - __uint_as_float(ah & 0xffff0000u), bl = b - __uint_as_float(bh & 0xffff0000u);
        lo[j] = __builtin_amdgcn_perm(__float_as_uint(bl), __float_as_uint(al), 0x07060302);
    }
}

// Places of one tile: group g (`groups`: rows of no adapter; -1: nothing) and [p0, p1).
struct Tile {
    int g, p0, p1, pad;
};

struct Groups {
    const int32_t *offsets, *order;
    int groups;
    int64_t rows;
    int32_t *dev_status;
};

__device__ __forceinline__ int wave_scan(int x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    return x;
}

// The slot-th tile of `high` places, counted group by group (rows of no group last); before:
// how many tiles of `small` places the groups before it have.  Wave uniform.
__device__ __forceinline__ Tile tile_of(const Groups &a, int high, int slot, int small, int &before) {
    const int lane = threadIdx.x & 63;
    before = 0;
    for (int base = 0; base <= a.groups; base += 64) {
        int64_t p = 0, z = 0;
        if (base + lane <= a.groups) rows_of_group(a.offsets, a.groups, a.rows, base + lane, p, z);
        const int mine = (int)((z - p + high - 1) / high), fine = (int)((z - p + small - 1) / small);
        const int upto = wave_scan(mine), fine_upto = wave_scan(fine);
        const uint64_t hit = __ballot(slot < upto);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            Tile t;
            t.g = base + src;
            const int first = __builtin_amdgcn_readlane((int)p, src), end = __builtin_amdgcn_readlane((int)z, src);
            t.p0 = first + (slot - __builtin_amdgcn_readlane(upto - mine, src)) * high;
            t.p1 = min(end, t.p0 + high);
            t.pad = 0;
            before += __builtin_amdgcn_readlane(fine_upto - fine, src);
            return t;
        }
        slot -= __builtin_amdgcn_readlane(upto, 63);
        before += __builtin_amdgcn_readlane(fine_upto, 63);
    }
    return {-1, 0, 0, 0};
}

// The row at a place; -1 past the tile and for one that is out of range.
__device__ __forceinline__ int row_at(const Groups &a, int place, int end) {
    if (place >= end) return -1;
    const int r = a.order ? a.order[place] : place;
    return r < 0 || r >= a.rows ? -1 : r;
}

// Offsets that fall or leave [0, rows], and places whose row is out of range, are reported.
__device__ __forceinline__ void report(const Groups &a, const Tile &t, bool first) {
    if (!a.dev_status) return;
    bool bad = false;
    if (first && a.offsets)
        for (int e = threadIdx.x; e < a.groups; e += blockDim.x) {
            const int p = a.offsets[e], z = a.offsets[e + 1];
            bad |= p < 0 || z < p || z > a.rows || (e == 0 && p != 0);
        }
    if (t.g >= 0 && a.order)
        for (int p = t.p0 + threadIdx.x; p < t.p1; p += blockDim.x) bad |= a.order[p] < 0 || a.order[p] >= a.rows;
    if (bad) atomicOr(a.dev_status, BAKRON_DEV_BAD_INDEX);
}

// ---------------------------------------------------------------- shrink

// One product of each of the two that a gradient needs: blockIdx.z.
struct Shrink {
    const char *x, *w;      // rows of K values; rank rows of K values a group
    int64_t ldx, ldw, group_w;
    int K;
    uint32_t *by_place;     // [16-place tile][16][ranks], or NULL
    uint32_t *by_rank;      // [16-place tile][ranks][16], or NULL
};
struct ShrinkArgs {
    Groups of;
    Shrink job[2];
    const float *scale;     // of a group, or NULL
    int rank, ranks;        // ranks: in whole 16s
    Tile *tiles;            // written by the first job
};

// The least tile is for few rows: its workgroup streams K with as many waves as fit.
constexpr int shrink_waves(int mt, int rt) { return mt == 1 && rt == 1 ? 16 : 8; }

template <int T, int MT, int RT>
__global__ __launch_bounds__(64 * shrink_waves(MT, RT)) void shrink_kernel(ShrinkArgs a) {
    extern __shared__ __align__(16) float space[];
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    constexpr int waves = shrink_waves(MT, RT);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = blockIdx.x, r0 = blockIdx.y * RT * 16;
    const Shrink &job = a.job[blockIdx.z];
    int before;
    const Tile t = tile_of(a.of, 16 * MT, slot, 16 * MT, before);
    if (blockIdx.y == 0 && blockIdx.z == 0) {
        if (threadIdx.x == 0) a.tiles[slot] = t;
        report(a.of, t, slot == 0);
    }
    if (t.g < 0 || t.g == a.of.groups) return;
    // Places past the tile and ranks past the last read a row that exists; their results
    // are not used.
    const char *x[MT], *m[RT];
    bool valid[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = row_at(a.of, t.p0 + i * 16 + l, t.p1);
        valid[i] = row >= 0;
        x[i] = job.x + 2 * max(row, 0) * job.ldx;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) m[i] = job.w + 2 * (t.g * job.group_w + min(r0 + i * 16 + l, a.rank - 1) * job.ldw);
    floatx4 acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
    // 64 of K a step: a wave reads whole lines
    const int whole = job.K / 64;
    uintx4 fx[2][MT], fm[2][RT];
    auto load = [&](int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = s * 64 + h * 32 + q * 8;
#pragma unroll
            for (int i = 0; i < MT; ++i) fx[h][i] = load_whole(x[i], k);
#pragma unroll
            for (int j = 0; j < RT; ++j) fm[h][j] = load_whole(m[j], k);
        }
    };
    auto multiply = [&](const uintx4(&gx)[2][MT], const uintx4(&gm)[2][RT]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[i][j] = mfma<T>(gx[h][i], gm[h][j], acc[i][j]);
    };
    if (w < whole) load(w);
    for (int s = w; s < whole; s += waves) {
        uintx4 gx[2][MT], gm[2][RT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) gx[h][i] = fx[h][i];
#pragma unroll
            for (int j = 0; j < RT; ++j) gm[h][j] = fm[h][j];
        }
        if (s + waves < whole) load(s + waves);
        multiply(gx, gm);
    }
    if (whole * 64 < job.K && w == whole % waves) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = whole * 64 + h * 32 + q * 8;
#pragma unroll
            for (int i = 0; i < MT; ++i) fx[h][i] = load_frag(x[i], k, job.K - k);
#pragma unroll
            for (int j = 0; j < RT; ++j) fm[h][j] = load_frag(m[j], k, job.K - k);
        }
        multiply(fx, fm);
    }
    // the waves' sums, in order
    floatx4 *sums = reinterpret_cast<floatx4 *>(space);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) sums[((i * RT + j) * waves + w) * 64 + lane] = acc[i][j];
    __syncthreads();
    const float scale = a.scale ? a.scale[t.g] : 1.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int c = i * RT + j;
            if (c % waves != w || r0 + j * 16 >= a.ranks) continue;
            floatx4 s = sums[c * waves * 64 + lane];
            for (int v = 1; v < waves; ++v) s += sums[(c * waves + v) * 64 + lane];
            // lane: rank l, places 4 q ..
            const int64_t tile = (int64_t)slot * MT + i;
            const int rank = r0 + j * 16 + l;
            uintx4 packed;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool ok = __shfl((int)valid[i], q * 4 + e) && rank < a.rank;
                packed[e] = ok ? pack_parts(s[e] * scale) : 0;
            }
            if (job.by_rank) *reinterpret_cast<uintx4 *>(job.by_rank + (tile * a.ranks + rank) * 16 + q * 4) = packed;
            if (job.by_place)
#pragma unroll
                for (int e = 0; e < 4; ++e) job.by_place[(tile * 16 + q * 4 + e) * a.ranks + rank] = packed[e];
        }
}

// ---------------------------------------------------------------- expand

struct ExpandArgs {
    Groups of;
    const Tile *tiles;
    const uint32_t *p;      // [16-place tile][16][ranks]
    const char *w;          // N rows of `rank` values a group
    int64_t group_w, ldw;
    const char *base;       // may be out; NULL: 0
    char *out;
    int64_t ldb, ldo;
    int N, rank, ranks, turns;  // turns: 64-column pieces of a wave
};

// 16 consecutive elements.
template <int T>
__device__ __forceinline__ void load16(const char *base, int64_t i, int left, float *x) {
    load8<T>(base, i, left, x);
    load8<T>(base, i + 8, left - 8, x + 8);
}
template <int T>
__device__ __forceinline__ void store16(char *base, int64_t i, int left, const float *x) {
    store8<T>(base, i, left, x);
    store8<T>(base, i + 8, left - 8, x + 8);
}

// D = W P^T with W's rows as the first operand: a lane then holds 4 of W's rows (columns of
// out) for one place.  The 64 columns of a piece are dealt to 4 products so that those are 16
// neighbours: row m of product t is column (m / 4) 16 + 4 t + m % 4.
template <int T, int OT, int MT, int RS>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs a) {
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pieces = (a.N + 63) / 64, per = 4 * a.turns, blocks = (pieces + per - 1) / per;
    const int64_t slot = blockIdx.x / blocks;
    const int block = (int)(blockIdx.x - slot * blocks);
    const Tile t = a.tiles[slot];
    if (t.g < 0) return;
    const bool none = t.g == a.of.groups;
    if (none && a.base == a.out) return;
    int row[MT];
    uintx4 hi[MT][RS], lo[MT][RS];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        row[i] = row_at(a.of, t.p0 + i * 16 + l, t.p1);
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            const int r = s * 32 + q * 8;
            uint32_t p[8] = {};
            if (!none && r < a.ranks) __builtin_memcpy(p, a.p + ((slot * MT + i) * 16 + l) * a.ranks + r, 32);
            unpack_parts(p, hi[i][s], lo[i][s]);
        }
    }
    for (int turn = 0; turn < a.turns; ++turn) {
        const int n0 = ((block * a.turns + turn) * 4 + w) * 64;
        if (n0 >= a.N) return;
        floatx4 acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = floatx4{0, 0, 0, 0};
        const int col = n0 + q * 16, left = a.N - col;
        float y[MT][16];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (a.base && row[i] >= 0) {
                load16<OT>(a.base, row[i] * a.ldb + col, left, y[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[i][e] = 0.0f;
            }
        }
        if (!none)
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                const int r = s * 32 + q * 8;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int n = min(n0 + (l >> 2) * 16 + c * 4 + (l & 3), a.N - 1);
                    const uintx4 f = load_frag(a.w, t.g * a.group_w + n * a.ldw + r, a.rank - r);
                    if constexpr (T == BAKRON_T_BF16) {
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            acc[i][c] = mfma_bf16(f, lo[i][s], mfma_bf16(f, hi[i][s], acc[i][c]));
                    } else {
                        uintx4 fh, fl;
                        split_f16(f, fh, fl);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc[i][c] = mfma_bf16(fh, lo[i][s], mfma_bf16(fh, hi[i][s], acc[i][c]));
                            acc[i][c] = mfma_bf16(fl, lo[i][s], mfma_bf16(fl, hi[i][s], acc[i][c]));
                        }
                    }
                }
            }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (row[i] < 0) continue;
            if (!none)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[i][c * 4 + e] += acc[i][c][e];
            store16<OT>(a.out, row[i] * a.ldo + col, left, y[i]);
        }
    }
}

// ---------------------------------------------------------------- transposes

// The gradients contract over the other dimension of A and B: rows x cols of each group
// that has rows, to cols x rows.
struct Transpose {
    const char *from;
    int64_t ld, group;
    char *to;
    int rows, cols;
};
struct TransposeArgs {
    Groups of;
    Transpose job[2];
};
__global__ __launch_bounds__(256) void transpose_kernel(TransposeArgs a) {
    __shared__ uint16_t tile[64][65];
    const Transpose &job = a.job[blockIdx.z];
    const int g = blockIdx.y, across = (job.cols + 63) / 64, down = (job.rows + 63) / 64;
    int64_t p, z;
    rows_of_group(a.of.offsets, a.of.groups, a.of.rows, g, p, z);
    if (p == z || blockIdx.x >= (unsigned)(across * down)) return;
    const int r0 = blockIdx.x / across * 64, c0 = blockIdx.x % across * 64;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const uint16_t *from = reinterpret_cast<const uint16_t *>(job.from) + g * job.group;
    uint16_t *to = reinterpret_cast<uint16_t *>(job.to) + (int64_t)g * job.rows * job.cols;
    for (int r = y; r < 64; r += 4)
        if (r0 + r < job.rows && c0 + x < job.cols) tile[r][x] = from[(r0 + r) * job.ld + c0 + x];
    __syncthreads();
    for (int c = y; c < 64; c += 4)
        if (c0 + c < job.cols && r0 + x < job.rows) to[(int64_t)(c0 + c) * job.rows + r0 + x] = tile[x][c];
}

// ---------------------------------------------------------------- outer

// G_g^T Z_g over a group's places: dA (rank x K, Z = X, G = U) or dB (N x rank, Z = dY, G = P).
struct Outer {
    const char *z;
    int64_t ldz;
    int cols;               // K or N
    const uint32_t *g;      // by_rank
    char *out;
    int64_t ldo, group_o;   // elements
    int by_column;          // dB: a row of `out` is one column of Z
    int64_t part0;          // first element of the job's partial sums in a unit's
};
struct OuterArgs {
    Groups of;
    Outer job[2];
    int rank, ranks, high;  // high: places of shrink's tiles
    int chunk, units;       // places of a unit; 0: a unit is a group
    int64_t subs;           // 16-place tiles that shrink has made
    int otype;
    float *part;            // [unit][part_size], with chunk
    int64_t part_size;
};

__device__ __forceinline__ void store_any(char *base, int type, int64_t i, int left, const float *x) {
    if (type == BAKRON_T_F32)
        store8<BAKRON_T_F32>(base, i, left, x);
    else if (type == BAKRON_T_BF16)
        store8<BAKRON_T_BF16>(base, i, left, x);
    else
        store8<BAKRON_T_F16>(base, i, left, x);
}
__device__ __forceinline__ void store_any1(char *base, int type, int64_t i, float x) {
    if (type == BAKRON_T_F32)
        store1<BAKRON_T_F32>(base, i, x);
    else if (type == BAKRON_T_BF16)
        store1<BAKRON_T_BF16>(base, i, x);
    else
        store1<BAKRON_T_F16>(base, i, x);
}

// A workgroup takes a unit's places, 128 columns and 16 RT ranks; its 4 waves share the
// places, 32 at a time.  A lane reads 8 columns of 8 rows and turns them about with byte
// permutes: the matrix cores want 8 places of one column.
template <int T, int RT>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs a) {
    __shared__ __align__(16) floatx4 space[2 * 8 * RT * 64];
    const Outer &job = a.job[blockIdx.z];
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int across = (job.cols + 127) / 128;
    const int unit = blockIdx.x % a.units, c0 = (blockIdx.x / a.units) * 128, r0 = blockIdx.y * RT * 16;
    if (c0 >= across * 128) return;
    Tile t;
    int before;
    if (a.chunk) {
        t = tile_of(a.of, a.chunk, unit, a.high, before);
        if (t.g < 0 || t.g == a.of.groups) return;
    } else {
        // all of group `unit`, also an empty one
        int64_t p, z;
        rows_of_group(a.of.offsets, a.of.groups, a.of.rows, unit, p, z);
        t = {unit, (int)p, (int)z, 0};
        before = 0;
        int sum = 0;
        for (int e = lane; e < unit; e += 64) {
            int64_t p2, z2;
            rows_of_group(a.of.offsets, a.of.groups, a.of.rows, e, p2, z2);
            sum += (int)((z2 - p2 + a.high - 1) / a.high);
        }
        before = __builtin_amdgcn_readlane(wave_scan(sum), 63);
    }
    int64_t p, z;
    rows_of_group(a.of.offsets, a.of.groups, a.of.rows, t.g, p, z);
    // shrink's 16-place tiles of this unit
    const int64_t sub = (int64_t)before * (a.high / 16) + (t.p0 - (int)p) / 16;
    const int col = c0 + l * 8, left = job.cols - col;
    floatx4 acc[8][RT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[c][r] = floatx4{0, 0, 0, 0};
    for (int s = w * 32; s < t.p1 - t.p0; s += 128) {
        uintx4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int row = row_at(a.of, t.p0 + s + q * 8 + e, t.p1);
            v[e] = row >= 0 ? load_frag(job.z, row * job.ldz + col, left) : uintx4{0, 0, 0, 0};
        }
        uintx4 gh[RT], gl[RT];
        const int64_t tile = sub + s / 16 + (q >> 1);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            uint32_t g[8] = {};
            const int rank = r0 + r * 16 + l;
            // past the unit's last 16-place tile there is none (nor where offsets fall)
            if (rank < a.ranks && tile >= 0 && tile < a.subs && t.p0 + s + (q & 2) * 8 < t.p1)
                __builtin_memcpy(g, job.g + (tile * a.ranks + rank) * 16 + (q & 1) * 8, 32);
            unpack_parts(g, gh[r], gl[r]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uintx4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __builtin_amdgcn_perm(v[2 * j + 1][c / 2], v[2 * j][c / 2], c & 1 ? 0x07060302 : 0x05040100);
            if constexpr (T == BAKRON_T_BF16) {
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[c][r] = mfma_bf16(f, gl[r], mfma_bf16(f, gh[r], acc[c][r]));
            } else {
                uintx4 fh, fl;
                split_f16(f, fh, fl);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    acc[c][r] = mfma_bf16(fh, gl[r], mfma_bf16(fh, gh[r], acc[c][r]));
                    acc[c][r] = mfma_bf16(fl, gl[r], mfma_bf16(fl, gh[r], acc[c][r]));
                }
            }
        }
    }
    // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
        if (w >= half && w < 2 * half)
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int r = 0; r < RT; ++r) space[(((w - half) * 8 + c) * RT + r) * 64 + lane] = acc[c][r];
        __syncthreads();
        if (w < half)
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[c][r] += space[((w * 8 + c) * RT + r) * 64 + lane];
        __syncthreads();
    }
    if (w != 0) return;
    // lane: rank l, columns 8 (4 q + e) + c
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int rank = r0 + r * 16 + l;
        if (rank >= a.rank) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = c0 + 8 * (4 * q + e);
            float x[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = acc[c][r][e];
            if (a.chunk) {
                store8<BAKRON_T_F32>(reinterpret_cast<char *>(a.part), unit * a.part_size + job.part0 + (int64_t)rank * job.cols + at,
                                     job.cols - at, x);
            } else if (!job.by_column) {
                store_any(job.out, a.otype, t.g * job.group_o + rank * job.ldo + at, job.cols - at, x);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (at + c < job.cols) store_any1(job.out, a.otype, t.g * job.group_o + (at + c) * job.ldo + rank, x[c]);
            }
        }
    }
}

// Adds a group's units, in order.  A thread takes 8 columns of a rank.
__global__ __launch_bounds__(256) void outer_join_kernel(OuterArgs a) {
    const Outer &job = a.job[blockIdx.z];
    const int g = blockIdx.y, per_row = (job.cols + 7) / 8;
    int first = 0;
    const int lane = threadIdx.x & 63;
    for (int e = lane; e < g; e += 64) {
        int64_t p, z;
        rows_of_group(a.of.offsets, a.of.groups, a.of.rows, e, p, z);
        first += (int)((z - p + a.chunk - 1) / a.chunk);
    }
    first = __builtin_amdgcn_readlane(wave_scan(first), 63);
    int64_t p, z;
    rows_of_group(a.of.offsets, a.of.groups, a.of.rows, g, p, z);
    const int last = min(a.units, first + (int)((z - p + a.chunk - 1) / a.chunk));
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.rank * per_row) return;
    const int rank = (int)(i / per_row), col = (int)(i - (int64_t)rank * per_row) * 8, left = job.cols - col;
    float sum[8] = {};
    for (int u = first; u < last; ++u) {
        float x[8];
        load8<BAKRON_T_F32>(reinterpret_cast<const char *>(a.part), u * a.part_size + job.part0 + (int64_t)rank * job.cols + col,
                            left, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += x[e];
    }
    if (!job.by_column) {
        store_any(job.out, a.otype, g * job.group_o + rank * job.ldo + col, left, sum);
    } else {
        for (int e = 0; e < 8 && e < left; ++e)
            store_any1(job.out, a.otype, g * job.group_o + (col + e) * job.ldo + rank, sum[e]);
    }
}

// ---------------------------------------------------------------- layout and launches

// How a call is laid out; the same for workspace and launch.
struct Layout {
    int mt, rt;             // shrink: 16-place tiles and 16-rank blocks of a workgroup
    int ranks, rs;          // ranks in whole 16s; 32-rank steps of expand
    int64_t slots;          // tiles of 16 mt places
    int chunk;              // of the sums over places; 0: a group is one unit
    int64_t units;
};

Layout layout_of(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups, bool grad) {
    Layout y;
    y.ranks = (int)round_up(rank, 16);
    y.rs = rank <= 32 ? 1 : rank <= 64 ? 2 : rank <= 128 ? 4 : 8;
    y.mt = rows >= 64 * (int64_t)(groups + 1) && rows >= 1024 ? 2 : 1;
    y.slots = row_tiles(16 * y.mt, rows, groups, true);
    const int blocks = y.ranks / 16;
    y.rt = y.slots * blocks <= 1024 ? 1 : blocks >= 4 ? 4 : blocks >= 2 ? 2 : 1;
    y.chunk = 0;
    y.units = groups;
    if (grad) {
        const int64_t tiles = (N + 127) / 128 + (K + 127) / 128, want = 1024;
        if (tiles * groups < want && rows > 512) {
            const int64_t splits = (want + tiles - 1) / tiles;
            y.chunk = (int)round_up((rows + splits - 1) / splits, 128);
            if (y.chunk < 256) y.chunk = 256;
            y.units = row_tiles(y.chunk, rows, groups, true);
        }
    }
    return y;
}

size_t place_words(const Layout &y) { return (size_t)y.slots * y.mt * 16 * y.ranks; }

template <int T, int MT, int RT>
void launch_shrink(const ShrinkArgs &a, const Layout &y, int jobs, hipStream_t s) {
    const dim3 grid((unsigned)y.slots, (unsigned)((y.ranks / 16 + RT - 1) / RT), jobs);
    hipLaunchKernelGGL((shrink_kernel<T, MT, RT>), grid, dim3(64 * shrink_waves(MT, RT)),
                       (size_t)shrink_waves(MT, RT) * MT * RT * 1024, s, a);
}
template <int T>
void launch_shrink(const ShrinkArgs &a, const Layout &y, int jobs, hipStream_t s) {
    if (y.mt == 1) {
        if (y.rt == 1) return launch_shrink<T, 1, 1>(a, y, jobs, s);
        if (y.rt == 2) return launch_shrink<T, 1, 2>(a, y, jobs, s);
        return launch_shrink<T, 1, 4>(a, y, jobs, s);
    }
    if (y.rt == 1) return launch_shrink<T, 2, 1>(a, y, jobs, s);
    if (y.rt == 2) return launch_shrink<T, 2, 2>(a, y, jobs, s);
    launch_shrink<T, 2, 4>(a, y, jobs, s);
}

int expand_turns(const Layout &y, int64_t N) {
    const int64_t pieces = (N + 63) / 64;
    int turns = 1;
    while (turns < 4 && y.slots * ((pieces + 8 * turns - 1) / (8 * turns)) >= 2048) turns *= 2;
    return turns;
}
int64_t expand_blocks(const Layout &y, int64_t N, int turns) { return y.slots * (((N + 63) / 64 + 4 * turns - 1) / (4 * turns)); }

template <int T, int OT, int MT>
void launch_expand(const ExpandArgs &a, const Layout &y, hipStream_t s) {
    const dim3 grid((unsigned)expand_blocks(y, a.N, a.turns));
    if (y.rs == 1)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 1>), grid, dim3(256), 0, s, a);
    else if (y.rs == 2)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 2>), grid, dim3(256), 0, s, a);
    else if (y.rs == 4)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 4>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 8>), grid, dim3(256), 0, s, a);
}
template <int T>
void launch_expand(ExpandArgs a, int32_t otype, const Layout &y, hipStream_t s) {
    a.turns = expand_turns(y, a.N);
    if (otype == BAKRON_T_F32)
        y.mt == 1 ? launch_expand<T, BAKRON_T_F32, 1>(a, y, s) : launch_expand<T, BAKRON_T_F32, 2>(a, y, s);
    else
        y.mt == 1 ? launch_expand<T, T, 1>(a, y, s) : launch_expand<T, T, 2>(a, y, s);
}

template <int T>
void launch_outer(const OuterArgs &a, const Layout &y, hipStream_t s) {
    const int64_t across = (std::max(a.job[0].cols, a.job[1].cols) + 127) / 128;
    const int blocks = y.ranks / 16;
    const unsigned x = (unsigned)(across * a.units);
    if (blocks == 1)
        hipLaunchKernelGGL((outer_kernel<T, 1>), dim3(x, 1, 2), dim3(256), 0, s, a);
    else if (blocks == 2)
        hipLaunchKernelGGL((outer_kernel<T, 2>), dim3(x, 1, 2), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((outer_kernel<T, 4>), dim3(x, (unsigned)((blocks + 3) / 4), 2), dim3(256), 0, s, a);
    if (a.chunk) {
        const int64_t threads = a.rank * across * 16;
        hipLaunchKernelGGL(outer_join_kernel, dim3((unsigned)((threads + 255) / 256), a.of.groups, 2), dim3(256), 0, s, a);
    }
}

bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool sizes_ok(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups) {
    if (!(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM && rank >= 1 &&
          rank <= MAX_RANK && groups >= 1 && groups <= MAX_GROUPS))
        return false;
    // no launch of 2^32 threads or more: the widest tiles' first dimension, in all of them
    const int64_t most = std::max(N, K), slots = row_tiles(16, rows, groups, true);
    return slots * 1024 <= LAUNCH_THREADS && slots * ((most + 255) / 256) * 256 <= LAUNCH_THREADS &&
           std::max<int64_t>(groups, 1024 + groups + 1) * ((most + 127) / 128) * 256 <= LAUNCH_THREADS &&
           ((most + 63) / 64) * ((rank + 63) / 64) * 256 <= LAUNCH_THREADS;
}

int32_t check_common(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups, const int32_t *offsets,
                     int32_t type) {
    BK_REQUIRE(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM,
               "bad sizes rows=%lld N=%lld K=%lld", (long long)rows, (long long)N, (long long)K);
    BK_REQUIRE(rank >= 1 && rank <= MAX_RANK, "rank must be in 1 .. %d, not %d", MAX_RANK, rank);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    BK_REQUIRE(sizes_ok(rows, N, K, rank, groups), "too many tiles: rows=%lld N=%lld K=%lld groups=%d", (long long)rows,
               (long long)N, (long long)K, groups);
    BK_REQUIRE(offsets || groups == 1, "offsets must be non-NULL for %d groups", groups);
    BK_REQUIRE(type == BAKRON_T_BF16 || type == BAKRON_T_F16, "type must be bf16 or fp16, not %d", type);
    return BAKRON_OK;
}

int32_t check_ld(const char *name, int64_t ld, int64_t width) {
    BK_REQUIRE(ld >= width && ld <= MAX_LD, "bad row stride %s=%lld for rows of %lld", name, (long long)ld,
               (long long)width);
    return BAKRON_OK;
}

int32_t check_out(const char *name, const void *p, int32_t otype, int32_t type) {
    BK_REQUIRE(otype == type || otype == BAKRON_T_F32, "the type of %s must be the inputs' or fp32, not %d", name, otype);
    BK_REQUIRE(aligned(p, elem_size(otype)), "%s is misaligned for its type", name);
    return BAKRON_OK;
}

int32_t check_ws(const void *ws, size_t have, size_t need) {
    if (ws && have >= need && aligned(ws, 256)) return BAKRON_OK;
    set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, have);
    return BAKRON_ERR_WORKSPACE;
}

size_t grad_size(const Layout &y, int64_t N, int64_t K, int32_t rank, int32_t groups, bool x, bool w) {
    size_t n = align256(y.slots * sizeof(Tile));
    n += align256((size_t)groups * rank * N * 2);                           // B^T
    if (x) n += align256((size_t)groups * rank * K * 2) + align256(place_words(y) * 4);  // A^T, U by place
    if (w) n += 2 * align256(place_words(y) * 4);                           // U and P by rank
    if (w && y.chunk) n += align256((size_t)y.units * rank * (N + K) * 4);
    return n;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

#define BK_TRY(expr)                          \
    do {                                      \
        int32_t bk_r_ = (expr);               \
        if (bk_r_ != BAKRON_OK) return bk_r_; \
    } while (0)

extern "C" size_t bakron_adapter_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t rank,
                                                       int32_t groups) {
    if (!sizes_ok(rows, N, K, rank, groups)) return 0;
    const Layout y = layout_of(rows, N, K, rank, groups, false);
    return align256(y.slots * sizeof(Tile)) + align256(place_words(y) * 4);
}

extern "C" int32_t bakron_adapter_matmul(const void *X, int32_t type, int64_t ldx, const void *A, const void *B,
                                         int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups,
                                         const int32_t *offsets, const int32_t *order, const float *scale,
                                         const void *base, int64_t ldb, void *out, int32_t otype, int64_t ldo,
                                         int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(X && A && B && out, "X, A, B and out must be non-NULL");
    BK_TRY(check_common(rows, N, K, rank, groups, offsets, type));
    BK_TRY(check_ld("ldx", ldx, K));
    BK_TRY(check_ld("ldo", ldo, N));
    if (base) BK_TRY(check_ld("ldb", ldb, N));
    BK_REQUIRE(base != out || ldb == ldo, "base in place of out has out's row stride");
    BK_REQUIRE(aligned(X, 2) && aligned(A, 2) && aligned(B, 2), "X, A or B is misaligned for its type");
    BK_TRY(check_out("out", out, otype, type));
    BK_TRY(check_out("base", base, otype, type));
    BK_TRY(check_ws(ws, ws_bytes, bakron_adapter_matmul_workspace_size(rows, N, K, rank, groups)));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    const Layout y = layout_of(rows, N, K, rank, groups, false);
    const Groups of = {offsets, order, groups, rows, dev_status};
    Carver c(ws);
    Tile *tiles = c.take<Tile>(y.slots);
    uint32_t *p = c.take<uint32_t>(place_words(y));
    ShrinkArgs h = {};
    h.of = of, h.scale = scale, h.rank = rank, h.ranks = y.ranks, h.tiles = tiles;
    h.job[0] = {static_cast<const char *>(X), static_cast<const char *>(A), ldx, K, rank * K, (int)K, p, nullptr};
    ExpandArgs e = {};
    e.of = of, e.tiles = tiles, e.p = p, e.w = static_cast<const char *>(B), e.group_w = N * rank, e.ldw = rank;
    e.base = static_cast<const char *>(base), e.out = static_cast<char *>(out), e.ldb = ldb, e.ldo = ldo;
    e.N = (int)N, e.rank = rank, e.ranks = y.ranks;
    if (type == BAKRON_T_BF16) {
        launch_shrink<BAKRON_T_BF16>(h, y, 1, s);
        launch_expand<BAKRON_T_BF16>(e, otype, y, s);
    } else {
        launch_shrink<BAKRON_T_F16>(h, y, 1, s);
        launch_expand<BAKRON_T_F16>(e, otype, y, s);
    }
    BK_LAUNCH_CHECK("adapter product");
    return BAKRON_OK;
}

extern "C" size_t bakron_adapter_matmul_grad_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t rank,
                                                            int32_t groups) {
    if (!sizes_ok(rows, N, K, rank, groups)) return 0;
    return grad_size(layout_of(rows, N, K, rank, groups, true), N, K, rank, groups, true, true);
}

extern "C" int32_t bakron_adapter_matmul_grad(const void *dY, int64_t lddy, const void *X, int32_t type, int64_t ldx,
                                              const void *A, const void *B, int64_t rows, int64_t N, int64_t K,
                                              int32_t rank, int32_t groups, const int32_t *offsets,
                                              const int32_t *order, const float *scale, const void *base, int64_t ldb,
                                              void *dX, int32_t xtype, int64_t lddx, void *dA, void *dB, int32_t wtype,
                                              int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(dY && A && B, "dY, A and B must be non-NULL");
    BK_REQUIRE(dX || (dA && dB), "dX, or dA and dB, must be non-NULL");
    BK_REQUIRE(!dA == !dB, "dA and dB go together");
    BK_REQUIRE(X || !dA, "dA and dB need X");
    BK_TRY(check_common(rows, N, K, rank, groups, offsets, type));
    BK_TRY(check_ld("lddy", lddy, N));
    if (dA) BK_TRY(check_ld("ldx", ldx, K));
    if (dX) {
        BK_TRY(check_ld("lddx", lddx, K));
        if (base) BK_TRY(check_ld("ldb", ldb, K));
        BK_REQUIRE(base != dX || ldb == lddx, "base in place of dX has dX's row stride");
        BK_TRY(check_out("dX", dX, xtype, type));
        BK_TRY(check_out("base", base, xtype, type));
    }
    if (dA) {
        BK_TRY(check_out("dA", dA, wtype, type));
        BK_TRY(check_out("dB", dB, wtype, type));
    }
    BK_REQUIRE(aligned(dY, 2) && aligned(X, 2) && aligned(A, 2) && aligned(B, 2),
               "dY, X, A or B is misaligned for its type");
    const Layout y = layout_of(rows, N, K, rank, groups, true);
    BK_TRY(check_ws(ws, ws_bytes, grad_size(y, N, K, rank, groups, dX, dA)));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    const Groups of = {offsets, order, groups, rows, dev_status};
    const char *x = static_cast<const char *>(X), *dy = static_cast<const char *>(dY);
    const char *a = static_cast<const char *>(A), *b = static_cast<const char *>(B);
    Carver c(ws);
    Tile *tiles = c.take<Tile>(y.slots);
    char *bt = c.take<char>((size_t)groups * rank * N * 2), *at = nullptr;
    uint32_t *u = nullptr, *ur = nullptr, *pr = nullptr;
    if (dX) at = c.take<char>((size_t)groups * rank * K * 2), u = c.take<uint32_t>(place_words(y));
    if (dA) ur = c.take<uint32_t>(place_words(y)), pr = c.take<uint32_t>(place_words(y));
    float *part = dA && y.chunk ? c.take<float>((size_t)y.units * rank * (N + K)) : nullptr;

    TransposeArgs t = {};
    t.of = of;
    t.job[0] = {b, rank, N * rank, bt, (int)N, rank};
    t.job[1] = {a, K, rank * K, at, rank, (int)K};
    const int64_t blocks = ((std::max(N, dX ? K : 1) + 63) / 64) * ((rank + 63) / 64);
    hipLaunchKernelGGL(transpose_kernel, dim3((unsigned)blocks, groups, dX ? 2 : 1), dim3(256), 0, s, t);

    ShrinkArgs h = {};
    h.of = of, h.scale = scale, h.rank = rank, h.ranks = y.ranks, h.tiles = tiles;
    h.job[0] = {dy, bt, lddy, N, rank * N, (int)N, u, ur};
    h.job[1] = {x, a, ldx, K, rank * K, (int)K, nullptr, pr};
    const int jobs = dA ? 2 : 1;
    type == BAKRON_T_BF16 ? launch_shrink<BAKRON_T_BF16>(h, y, jobs, s) : launch_shrink<BAKRON_T_F16>(h, y, jobs, s);

    if (dX) {
        ExpandArgs e = {};
        e.of = of, e.tiles = tiles, e.p = u, e.w = at, e.group_w = K * rank, e.ldw = rank;
        e.base = static_cast<const char *>(base), e.out = static_cast<char *>(dX), e.ldb = ldb, e.ldo = lddx;
        e.N = (int)K, e.rank = rank, e.ranks = y.ranks;
        type == BAKRON_T_BF16 ? launch_expand<BAKRON_T_BF16>(e, xtype, y, s) : launch_expand<BAKRON_T_F16>(e, xtype, y, s);
    }
    if (dA) {
        OuterArgs o = {};
        o.of = of, o.rank = rank, o.ranks = y.ranks, o.high = 16 * y.mt, o.chunk = y.chunk, o.units = (int)y.units;
        o.subs = y.slots * y.mt;
        o.otype = wtype, o.part = part, o.part_size = (int64_t)rank * (N + K);
        o.job[0] = {x, ldx, (int)K, ur, static_cast<char *>(dA), K, rank * K, 0, 0};
        o.job[1] = {dy, lddy, (int)N, pr, static_cast<char *>(dB), rank, N * rank, 1, rank * K};
        type == BAKRON_T_BF16 ? launch_outer<BAKRON_T_BF16>(o, y, s) : launch_outer<BAKRON_T_F16>(o, y, s);
    }
    BK_LAUNCH_CHECK("adapter gradients");
    return BAKRON_OK;
}
