// products.hip -- bakron_fp8_matmul, bakron_grouped_matmul and its gradients.
//
// All are one tiled product C[i][j] = sum_r P[i][r] Q[j][r] on the matrix cores,
// for rows i that belong to groups (experts) of ragged sizes:
//   forward      P = X (rows x K),  Q = W_g (N x K),          both r-contiguous
//   gradient X   P = dY (rows x N), Q = W_g as [r = n][j = k], r strided
//   gradient W   per group, r runs over its rows: P = dY as [r][i = n],
//                Q = X as [r][j = k], both r strided
// fp8 operands carry a scale for each 128 of r, so their products of one K step
// are summed by themselves and then added with the scale, in fp32.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "elem.hpp"
#include "walk.hpp"

namespace bakron {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

enum { F8 = 3 };                                        // element type beside BAKRON_T_*
enum { SCALE_NONE = -1 };                               // else BAKRON_SCALE_*
enum { FWD = 0, GRAD_X = 1, GRAD_W = 2 };

constexpr int STEP = 128;  // bytes of r in one K step of an r-contiguous operand

struct ProductArgs {
    const char *P, *Q;
    char *Y;
    int64_t ldp, ldq;        // bytes
    int64_t ldy;             // elements
    int64_t group_q;         // bytes from a group's Q to the next (forward, gradient X)
    int64_t group_y;         // elements from a group's C to the next (gradient W)
    const float *sp, *sq;    // fp8 scales
    int64_t rows, I, J, R;   // rows: of all groups; I: gradient W's row count; R: forward, gradient X
    int groups;
    const int32_t *offsets;  // NULL: one group of all rows
    int32_t *dev_status;
    int ytype;
    int tiles_i, tiles_j;    // tiles_i: gradient W
    int slots;               // row tiles that launch and workspace are sized for (forward, gradient X)
    int vec;                 // 1: rows of C start on 16 bytes
    int splits;              // parts of the reduction, each a workgroup of its own
    float *part;             // with splits > 1: the parts' sums, as the accumulators hold them
    int tail;                // 1: large tiles leave their tail to small ones
    unsigned large;          // workgroups of large tiles, before those of a tail in their launch
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int64_t uniform(int64_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

// Sum of a lane's value and those of the lanes below it.  Rows of 16 lanes are
// scanned first, then the rows' totals are passed on.
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // from 1 lane below in the row
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, true);   // lane 15's to row 1, 47's to row 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, true);   // lane 31's to rows 2 and 3
    return x;
}

__device__ __forceinline__ void group_range(const ProductArgs &p, int g, int64_t &a, int64_t &b) {
    rows_of_group(p.offsets, p.groups, p.rows, g, a, b);
}

// Offsets that fall or leave [0, rows] are reported once.
__device__ __forceinline__ void report_offsets(const ProductArgs &p) {
    if (blockIdx.x != 0 || threadIdx.x >= 64 || !p.offsets || !p.dev_status) return;
    bool bad = false;
    for (int e = threadIdx.x; e < p.groups; e += 64) {
        const int a = p.offsets[e], b = p.offsets[e + 1];
        bad |= a < 0 || b < a || b > p.rows || (e == 0 && a != 0);
    }
    if (bad) atomicOr(p.dev_status, BAKRON_DEV_BAD_INDEX);
}

constexpr unsigned TAIL_MOST = 4 * 128;  // workgroups of a tail (without_tail)

// Finds the workgroup's rows: tiles of BI rows are counted group by group, then
// walked in bands of 8 row tiles.  All 64 lanes of a wave take part; the results are
// wave uniform.  False: no work for this workgroup.
template <int BI>
__device__ __forceinline__ bool find_rows(const ProductArgs &p, int64_t b, bool tail, int &g, int64_t &i0, int64_t &i1,
                                          int &tj, int64_t &w) {
    const int lane = threadIdx.x & 63;
    // lane e holds group e's first row and tiles, for the first 64 groups
    int first = 0, mine = 0, upto = 0, slots;
    int64_t a, z;
    auto tiles_of = [&](int e) {
        a = z = 0;
        if (e <= p.groups) group_range(p, e, a, z);
        return (int)((z - a + BI - 1) / BI);
    };
    if (!p.offsets) {
        slots = (int)((p.rows + BI - 1) / BI);
    } else {
        mine = tiles_of(lane);
        first = (int)a;
        upto = wave_scan(mine);
        slots = __builtin_amdgcn_readlane(upto, 63);
        for (int base = 64; base <= p.groups; base += 64)
            slots += __builtin_amdgcn_readlane(wave_scan(tiles_of(base + lane)), 63);
    }
    int slot;
    if (!place_of(slots, p.slots, p.tiles_j, p.tail, tail, b, w, slot, tj)) return false;
    tj = (int)uniform(tj);
    slot = (int)uniform(slot);
    if (!p.offsets) {
        g = 0;
        i0 = (int64_t)slot * BI;
        i1 = min<int64_t>(p.rows, i0 + BI);
        return true;
    }
    for (int base = 0;;) {
        const uint64_t hit = __ballot(slot < upto);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int before = __builtin_amdgcn_readlane(upto - mine, src);
            g = base + src;
            const int at = __builtin_amdgcn_readlane(first, src);
            group_range(p, g, a, z);
            i0 = at + (int64_t)(slot - before) * BI;
            i1 = min<int64_t>(uniform(z), i0 + BI);
            return true;
        }
        slot -= __builtin_amdgcn_readlane(upto, 63);
        base += 64;
        if (base > p.groups) return false;
        mine = tiles_of(base + lane);
        first = (int)a;
        upto = wave_scan(mine);
    }
}

// A workgroup's part of the product; all wave uniform.
struct Work {
    int g, tj, s0;      // group, column tile, first step of the reduction
    int64_t i0, i1, R;  // rows of C, length of the reduction
    const char *P, *Q;  // at the group's first row and the reduction's start
    int64_t yoff;       // elements before the group's C
    int64_t nth;        // number of the tile and part
};

template <int MODE, int BI, int KR>
__device__ __forceinline__ bool find_work(const ProductArgs &p, unsigned block, bool tail, Work &t) {
    report_offsets(p);
    // in the tail, four workgroups of one XCD share a large tile
    constexpr int LARGE = 256;
    const int64_t b = tail ? (block >> 5 << 3) + (block & 7) : block / p.splits;
    const int part = tail ? 0 : block % p.splits, quarter = tail ? block >> 3 & 3 : 0;
    const int size = tail ? LARGE : BI;
    t.P = p.P, t.Q = p.Q, t.R = p.R, t.yoff = 0;
    int64_t w;
    if constexpr (MODE == GRAD_W) {
        const int64_t tiles = (int64_t)p.tiles_i * p.tiles_j, total = tiles * p.groups;
        const int64_t most = p.tail ? without_tail(total) : total, at = tail ? most + b : b;
        if (at >= (tail ? total : most)) return false;
        // every XCD gets a part of each group's tiles: groups differ in length (8192 rows
        // in 16 uneven groups, both gradients: 0.41 against 0.45 ms)
        t.g = (int)(at / tiles);
        const int n = (int)xcd_order(at - t.g * tiles, tiles);
        w = t.g * tiles + n;
        // in bands of 4 rows of tiles: an XCD's part is about square, so its L2 fetches
        // less (135 against 280 MB there, 0.38 against 0.39 ms)
        const int band = n / (4 * p.tiles_j), left = n - band * 4 * p.tiles_j;
        const int high = min(4, p.tiles_i - band * 4);
        t.tj = left / high;
        t.i0 = (int64_t)(band * 4 + left % high) * size;
        t.i1 = min<int64_t>(p.I, t.i0 + size);
        int64_t a, z;
        group_range(p, t.g, a, z);
        a = uniform(a);
        t.R = uniform(z) - a;
        t.P += a * p.ldp;
        t.Q += a * p.ldq;
        t.yoff = t.g * p.group_y;
    } else {
        if (tail ? !find_rows<LARGE>(p, b, true, t.g, t.i0, t.i1, t.tj, w)
                 : !find_rows<BI>(p, b, false, t.g, t.i0, t.i1, t.tj, w))
            return false;
        t.g = (int)uniform(t.g), t.tj = (int)uniform(t.tj);
        t.i0 = uniform(t.i0), t.i1 = uniform(t.i1);
        if (t.g == p.groups)
            t.R = 0;  // rows of no group
        else
            t.Q += t.g * p.group_q;
    }
    if (tail) {
        t.i0 += quarter % 2 * BI;
        t.i1 = min<int64_t>(t.i1, t.i0 + BI);
        t.tj = t.tj * (LARGE / BI) + quarter / 2;
        if (t.i0 >= t.i1 || (int64_t)t.tj * BI >= p.J) return false;
    }
    t.nth = uniform(w) * p.splits + part;
    t.s0 = 0;
    if (p.splits > 1) {
        const int steps = (int)((t.R + KR - 1) / KR);
        t.s0 = (int)uniform((int64_t)steps * part / p.splits);
        const int s1 = (int)uniform((int64_t)steps * (part + 1) / p.splits);
        t.P += MODE == GRAD_W ? (int64_t)t.s0 * KR * p.ldp : (int64_t)t.s0 * STEP;
        t.Q += MODE != FWD ? (int64_t)t.s0 * KR * p.ldq : (int64_t)t.s0 * STEP;
        t.R = min<int64_t>(t.R, (int64_t)s1 * KR) - (int64_t)t.s0 * KR;
    }
    return true;
}

// 16 bytes of an operand: `left` elements of ES bytes are there, the rest is 0.
template <int ES>
__device__ __forceinline__ intx4 chunk(const char *src, int64_t left) {
    intx4 v = {0, 0, 0, 0};
    if (left >= 16 / ES) {
        __builtin_memcpy(&v, src, 16);
    } else if (left > 0) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 16 / ES; ++q)
            if (q < left) {
                if constexpr (ES == 1)
                    w[q / 4] |= (uint32_t)reinterpret_cast<const uint8_t *>(src)[q] << (8 * (q % 4));
                else
                    w[q / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[q] << (16 * (q % 2));
            }
        v = intx4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
    return v;
}

// One operand's tile in LDS, for one K step.
//  r contiguous: BC rows of 128 bytes; 16-byte chunk c of row n at place
//    c ^ (n & 7), so that 8 rows' reads of one chunk touch all banks.
//  r strided: 64 rows of r, each BC 16-bit columns; the 32-byte unit u (16
//    columns) of row r at place u ^ swap(r), so that the 4 rows that a
//    transposing read joins, and those of its neighbours, lie in other banks.
template <int ET, bool STRIDED, int BC>
struct Tile {
    static constexpr int ES = ET == F8 ? 1 : 2;
    static constexpr int BYTES = BC * STEP;
    static constexpr int CHUNKS = BYTES / 16;
    static constexpr int ROW = STRIDED ? BC * 2 : STEP;  // bytes of a row in LDS
    static __device__ __forceinline__ int swap(int r) {
        return STRIDED ? (r & 3) | ((r >> 1) & 4) : r & 7;
    }

    // where the chunk at LDS place q comes from: row (of the tile, or of r) and byte in it
    static __device__ __forceinline__ void place(int q, int &row, int &byte) {
        row = q / (ROW / 16);
        const int c = q % (ROW / 16);
        if constexpr (STRIDED)
            byte = (((c >> 1) ^ swap(row)) << 5) | ((c & 1) << 4);
        else
            byte = (c ^ swap(row)) << 4;
    }

    // byte address of the lane's first 8 bytes (strided) or 16 bytes for tile columns
    // c0 .. c0 + 15 and part h of r (32 values of 2 bytes, or 64 of 1)
    static __device__ __forceinline__ int frag(int c0, int h, int lane) {
        const int l = lane & 15, g = lane >> 4;
        if constexpr (STRIDED) {
            const int r = 32 * h + 8 * g + (l >> 2);
            return r * ROW + (((c0 >> 4) ^ swap(r)) << 5) + (l & 3) * 8;
        } else {
            const int n = c0 + l;
            return n * STEP + (((4 * h + g) ^ swap(n)) << 4);
        }
    }
    static __device__ __forceinline__ intx4 read(const char *lds, int c0, int h, int lane) {
        const char *src = lds + frag(c0, h, lane);
        if constexpr (STRIDED) {
            // lane l of 16 gets column c0 + l and 4 rows of r from each read
            typedef __attribute__((address_space(3))) shortx4 *lp;
            const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(src));
            const shortx4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(src + 4 * ROW));
            struct { shortx4 a, b; } v = {a, b};
            intx4 r;
            __builtin_memcpy(&r, &v, 16);
            return r;
        } else {
            return *reinterpret_cast<const intx4 *>(src);
        }
    }
};

template <int ET>
__device__ __forceinline__ floatx4 mfma(intx4 a, intx4 b, floatx4 c) {
    if constexpr (ET == BAKRON_T_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// The same in place, on accumulation registers.  Written out because the compiler
// moves accumulators about when they fill all 256 of these registers.  It does not
// see the hazards of this form: settle() stands between other accesses of the
// accumulators and these products, in both directions.  That nothing else comes too
// close is checked in the assembly that is compiled (tests/test_products_assembly.py).
template <int ET>
__device__ __forceinline__ void mfma_in_place(intx4 a, intx4 b, floatx4 &c) {
    if constexpr (ET == BAKRON_T_BF16)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

__device__ __forceinline__ floatx4 mfma_f8(intx4 a0, intx4 a1, intx4 b0, intx4 b1) {
    const intx8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const intx8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    const floatx4 zero = {0, 0, 0, 0};
    // format 0 = e4m3 on both sides; all block exponents 2^0
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// A wave's part of a tile, NI x NJ accumulators: rows from i0 on (below i1), columns
// from j0 on.  An accumulator's lane holds 4 columns of one row, so stores from there
// would touch a quarter of a line each; the part goes through LDS (`scratch`, 512 NI NJ
// bytes of this wave's own; fp32 results in two turns, half of the columns each) and
// leaves as whole rows, 16 bytes a lane.  The 16-byte chunk c of row r lies at place
// c ^ r.  One wait between the writes and the reads of a turn: with 4 waves a CU there
// is little else to run meanwhile (16 rows at a time took twice as long).  PAST: large
// tiles' results go past the caches, which keep the operands (gradients of 8192 rows by
// 16 groups of 4096 x 2048: 0.36 against 0.38 ms; 27 MB of results from small tiles are
// slower that way, 34.6 against 33.4 us).
template <int SCALE, int NI, int NJ, bool PAST>
__device__ __forceinline__ void store_tile(const ProductArgs &p, floatx4 (&acc)[NI][NJ], int g, int64_t yoff,
                                           int64_t i0, int64_t i1, int64_t j0, int lane, char *scratch) {
    constexpr int CH = 2 * NJ, ROWS = 64 / CH;  // chunks of a row, rows a wave stores at once
    static_assert((NJ & (NJ - 1)) == 0 && NJ >= 2 && NJ <= 8, "a power of two chunks a row, at most 16");
    const int l = lane & 15, q = lane >> 4;
    const bool f32 = p.ytype == BAKRON_T_F32;
    const int es = f32 ? 4 : 2, per = 16 / es;
    // the scales of the wave's columns, one a lane and 64 columns
    float w[(NJ + 3) / 4];
    if constexpr (SCALE == BAKRON_SCALE_ROW)
#pragma unroll
        for (int k = 0; k < (NJ + 3) / 4; ++k) {
            const int64_t j = j0 + 64 * k + lane;
            w[k] = g < p.groups && j < p.J ? p.sq[g * p.J + j] : 0.0f;
        }
    auto write = [&](auto type, int b0, int b1) __attribute__((always_inline)) {
        constexpr int T = decltype(type)::value;
#pragma unroll
        for (int b = 0; b < NJ; ++b) {
            if (b < b0 || b >= b1) continue;
            float ws[4];
            if constexpr (SCALE == BAKRON_SCALE_ROW)
#pragma unroll
                for (int v = 0; v < 4; ++v) ws[v] = __shfl(w[b / 4], (b % 4) * 16 + 4 * q + v);
            const int k = T == BAKRON_T_F32 ? 4 * (b - b0) + q : 2 * b + (q >> 1);
            char *to = scratch + l * CH * 16 + ((k ^ l) & (CH - 1)) * 16 + (T == BAKRON_T_F32 ? 0 : (q & 1) * 8);
#pragma unroll
            for (int a = 0; a < NI; ++a) {
                floatx4 t = acc[a][b];
                if constexpr (SCALE == BAKRON_SCALE_ROW)
#pragma unroll
                    for (int v = 0; v < 4; ++v) t[v] *= ws[v];
                if constexpr (T == BAKRON_T_F32)
                    *reinterpret_cast<floatx4 *>(to + a * 16 * CH * 16) = t;
                else
                    *reinterpret_cast<uint2 *>(to + a * 16 * CH * 16) = make_uint2(pack2<T>(t[0], t[1]), pack2<T>(t[2], t[3]));
            }
        }
    };
    const int c = lane % CH, r0 = lane / CH;
    const bool full = p.vec && i0 + 16 * NI <= i1 && j0 + 16 * NJ <= p.J;
    const int64_t down = (int64_t)ROWS * p.ldy * es;
    auto leave = [&](int turn) __attribute__((always_inline)) {
        // the wave's own writes, then reads: in order, no other wave takes part
        __builtin_amdgcn_wave_barrier();
        const int64_t jc = j0 + turn * NJ * 8 + c * per;
        char *y = p.Y + (yoff + (i0 + r0) * p.ldy + jc) * es;
        const char *from = scratch + r0 * CH * 16;
        if (full) {
#pragma unroll 4
            for (int r = r0; r < 16 * NI; r += ROWS, from += ROWS * CH * 16, y += down) {
                const intx4 v = *reinterpret_cast<const intx4 *>(from + ((c ^ r) & (CH - 1)) * 16);
                if constexpr (PAST)
                    __builtin_nontemporal_store(v, reinterpret_cast<intx4 *>(y));
                else
                    *reinterpret_cast<intx4 *>(y) = v;
            }
        } else {
            const int left = (int)min<int64_t>(per, p.J - jc), rows = (int)min<int64_t>(16 * NI, i1 - i0);
#pragma unroll 1
            for (int r = r0; r < rows; r += ROWS, from += ROWS * CH * 16, y += down) {
                const intx4 v = *reinterpret_cast<const intx4 *>(from + ((c ^ r) & (CH - 1)) * 16);
                if (left == per && p.vec) {
                    *reinterpret_cast<intx4 *>(y) = v;
                } else if (f32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) reinterpret_cast<int *>(y)[e] = v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) reinterpret_cast<uint16_t *>(y)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    };
    if (f32) {
        write(std::integral_constant<int, BAKRON_T_F32>(), 0, NJ / 2);
        leave(0);
        write(std::integral_constant<int, BAKRON_T_F32>(), NJ / 2, NJ);
        leave(1);
    } else {
        if (p.ytype == BAKRON_T_BF16)
            write(std::integral_constant<int, BAKRON_T_BF16>(), 0, NJ);
        else
            write(std::integral_constant<int, BAKRON_T_F16>(), 0, NJ);
        leave(0);
    }
}

// A part's sums, register by register.
template <int NI, int NJ>
__device__ __forceinline__ void store_part(float *part, floatx4 (&acc)[NI][NJ], int wave, int lane) {
    floatx4 *to = reinterpret_cast<floatx4 *>(part) + wave * NI * NJ * 64 + lane;
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int b = 0; b < NJ; ++b) to[(a * NJ + b) * 64] = acc[a][b];
}

// Adds the parts of each tile in their order and stores it.  A wave takes 16 of a
// tile's 256 accumulators: 16 rows by 64 columns; PIECES waves, each a workgroup,
// share a tile, as few tiles are what the parts are for.
constexpr int PIECES = 16;
template <int MODE, int SCALE, int KR>
__global__ __launch_bounds__(64) void product_join_kernel(ProductArgs p, int parts) {
    constexpr int BI = 128, BJ = 128, NI = 4, NJ = 4;
    __shared__ __align__(16) char lds[512 * NJ];
    const int lane = threadIdx.x;
    Work t;
    p.splits = PIECES;
    if (!find_work<MODE, BI, KR>(p, blockIdx.x, false, t)) return;
    const int64_t tile = t.nth / PIECES;
    const int piece = (int)(t.nth % PIECES), wave = piece / NI, a = piece % NI;
    floatx4 acc[1][NJ];
    const floatx4 *from = reinterpret_cast<const floatx4 *>(p.part) + tile * parts * (BI * BJ / 4) +
                          (wave * NI + a) * NJ * 64 + lane;
#pragma unroll
    for (int b = 0; b < NJ; ++b) acc[0][b] = from[b * 64];
#pragma unroll 4
    for (int k = 1; k < parts; ++k) {
        from += BI * BJ / 4;
#pragma unroll
        for (int b = 0; b < NJ; ++b) acc[0][b] += from[b * 64];
    }
    store_tile<SCALE, 1, NJ, false>(p, acc, t.g, t.yoff, t.i0 + wave % 2 * 64 + a * 16, t.i1,
                             (int64_t)t.tj * BJ + wave / 2 * 64, lane, lds);
}

// One BI x BJ tile of C by WI x WJ waves; K steps are staged through registers
// (any alignment, any sizes), the next step's loads in flight during a step.
// Accumulators: lane l holds row i = l % 16 and columns j = 4 (l / 16) + v.
template <int ET, int MODE, int SCALE, int BI, int BJ, int WI, int WJ>
__global__ __launch_bounds__(64 * WI * WJ) void product_kernel(ProductArgs p) {
    constexpr bool PS = MODE == GRAD_W, QS = MODE != FWD;
    typedef Tile<ET, PS, BI> TP;
    typedef Tile<ET, QS, BJ> TQ;
    constexpr int ES = TP::ES, KR = STEP / ES;  // bytes of an element, values of r in a step
    constexpr int NTH = 64 * WI * WJ, CP = TP::CHUNKS / NTH, CQ = TQ::CHUNKS / NTH;
    constexpr int NI = BI / WI / 16, NJ = BJ / WJ / 16;
    __shared__ __align__(16) char lds[TP::BYTES + TQ::BYTES];
    char *const lp = lds, *const lq = lds + TP::BYTES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave % WI, wj = wave / WI;

    Work t;
    if (!find_work<MODE, BI, KR>(p, blockIdx.x, false, t)) return;
    const int g = t.g;
    const int64_t i0 = t.i0, i1 = t.i1, j0 = (int64_t)t.tj * BJ, R = t.R, yoff = t.yoff;
    const char *P = t.P, *Q = t.Q;
    const int steps = (int)((R + KR - 1) / KR);

    intx4 rp[CP], rq[CQ];
    auto load = [&](int s) {
        const int64_t r0 = (int64_t)s * KR;
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            int row, byte;
            TP::place(tid + c * NTH, row, byte);
            if constexpr (PS)
                rp[c] = chunk<ES>(P + (r0 + row) * p.ldp + i0 * ES + byte, r0 + row < R ? p.I - i0 - byte / ES : 0);
            else
                rp[c] = chunk<ES>(P + (i0 + row) * p.ldp + r0 * ES + byte, i0 + row < i1 ? R - r0 - byte / ES : 0);
        }
#pragma unroll
        for (int c = 0; c < CQ; ++c) {
            int row, byte;
            TQ::place(tid + c * NTH, row, byte);
            if constexpr (QS)
                rq[c] = chunk<ES>(Q + (r0 + row) * p.ldq + j0 * ES + byte, r0 + row < R ? p.J - j0 - byte / ES : 0);
            else
                rq[c] = chunk<ES>(Q + (j0 + row) * p.ldq + r0 * ES + byte, j0 + row < p.J ? R - r0 - byte / ES : 0);
        }
    };

    floatx4 acc[NI][NJ];
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int b = 0; b < NJ; ++b) acc[a][b] = floatx4{0, 0, 0, 0};

    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CP; ++c) *reinterpret_cast<intx4 *>(lp + (tid + c * NTH) * 16) = rp[c];
#pragma unroll
        for (int c = 0; c < CQ; ++c) *reinterpret_cast<intx4 *>(lq + (tid + c * NTH) * 16) = rq[c];
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
        if constexpr (ET == F8) {
            float sc[NI];
#pragma unroll
            for (int a = 0; a < NI; ++a) {
                const int64_t i = i0 + wi * (BI / WI) + a * 16 + (lane & 15);
                sc[a] = p.sp[(t.s0 + s) * p.rows + min<int64_t>(i, i1 - 1)];
            }
            if constexpr (SCALE == BAKRON_SCALE_BLOCK) {
                // a wave's columns lie in one block of 128
                const int64_t nb = (p.J + 127) / 128;
                const int64_t jb = min<int64_t>((j0 + wj * (BJ / WJ)) / 128, nb - 1);
                const float w = p.sq[((int64_t)g * ((p.R + KR - 1) / KR) + t.s0 + s) * nb + jb];
#pragma unroll
                for (int a = 0; a < NI; ++a) sc[a] *= w;
            }
            intx4 fp[NI][2];
#pragma unroll
            for (int a = 0; a < NI; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) fp[a][h] = TP::read(lp, wi * (BI / WI) + a * 16, h, lane);
#pragma unroll
            for (int b = 0; b < NJ; ++b) {
                const intx4 q0 = TQ::read(lq, wj * (BJ / WJ) + b * 16, 0, lane);
                const intx4 q1 = TQ::read(lq, wj * (BJ / WJ) + b * 16, 1, lane);
#pragma unroll
                for (int a = 0; a < NI; ++a) {
                    const floatx4 sum = mfma_f8(q0, q1, fp[a][0], fp[a][1]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[a][b][v] = fmaf(sc[a], sum[v], acc[a][b][v]);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                intx4 fp[NI];
#pragma unroll
                for (int a = 0; a < NI; ++a) fp[a] = TP::read(lp, wi * (BI / WI) + a * 16, h, lane);
#pragma unroll
                for (int b = 0; b < NJ; ++b) {
                    const intx4 fq = TQ::read(lq, wj * (BJ / WJ) + b * 16, h, lane);
#pragma unroll
                    for (int a = 0; a < NI; ++a) acc[a][b] = mfma<ET>(fq, fp[a], acc[a][b]);
                }
            }
        }
    }

    if (p.splits > 1) {
        store_part<NI, NJ>(p.part + t.nth * BI * BJ, acc, wave, lane);
        return;
    }
    // every wave is done with the operands' buffers, which now carry the results
    static_assert(512 * NI * NJ * WI * WJ <= (int)sizeof(lds), "the results of each wave");
    __syncthreads();
    store_tile<SCALE, NI, NJ, false>(p, acc, g, yoff, i0 + wi * (BI / WI), i1, j0 + wj * (BJ / WJ), lane,
                              lds + wave * 512 * NI * NJ);
}

// 16 zero bytes: what a lane loads in the place of r beyond the end.
__device__ const uint4 zero_chunk = {0, 0, 0, 0};

// Loads 16 bytes a lane straight into LDS, lane l's at `lds` + 16 l (wave uniform).
// The wait for them is stage_wait's: the compiler does not count these loads.  m0 is the
// compiler's own and cannot be declared; it has no use for it in these kernels, which is
// checked with the rest of the assembly, as is the distance from what computes `base`.
__device__ __forceinline__ void load_lds(const char *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void load_lds(const char *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds)
                 : "memory");
}
// All but this wave's last N loads have arrived and its LDS reads are done; then
// every wave's.
template <int N = 0>
__device__ __forceinline__ void stage_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The same product for operands whose rows begin on 16 bytes and whose widths are
// whole 16-byte chunks: each step's tiles go straight from memory to LDS, into the
// others of NB buffers while a step is computed.
// `lds` holds NB steps of both operands.
template <int ET, int MODE, int SCALE, int BI, int BJ, int WI, int WJ, int NB>
__device__ __forceinline__ void direct_tile(const ProductArgs &p, unsigned block, bool tail, char *lds) {
    constexpr bool PS = MODE == GRAD_W, QS = MODE != FWD;
    typedef Tile<ET, PS, BI> TP;
    typedef Tile<ET, QS, BJ> TQ;
    constexpr int ES = TP::ES, KR = STEP / ES;
    constexpr int NTH = 64 * WI * WJ, CP = TP::CHUNKS / NTH, CQ = TQ::CHUNKS / NTH;
    constexpr int NI = BI / WI / 16, NJ = BJ / WJ / 16;
    constexpr int BUF = TP::BYTES + TQ::BYTES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave % WI, wj = wave / WI;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;

    Work t;
    if (!find_work<MODE, BI, KR>(p, block, tail, t)) return;
    const int g = t.g;
    const int64_t i0 = t.i0, i1 = t.i1, j0 = (int64_t)t.tj * BJ, R = t.R, yoff = t.yoff;
    const char *P = t.P, *Q = t.Q;
    const int steps = __builtin_amdgcn_readfirstlane((int)((R + KR - 1) / KR));

    // Where this lane's chunks come from, relative to the tile's first.  Rows and
    // columns past the edge repeat the last ones (their results are not stored).
    uint32_t op[CP], oq[CQ];
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        int row, byte;
        TP::place(tid + c * NTH, row, byte);
        if constexpr (PS)
            op[c] = (uint32_t)(row * p.ldp + min<int64_t>(byte, (p.I - i0) * ES - 16));
        else
            op[c] = (uint32_t)(min<int64_t>(row, i1 - i0 - 1) * p.ldp + byte);
    }
#pragma unroll
    for (int c = 0; c < CQ; ++c) {
        int row, byte;
        TQ::place(tid + c * NTH, row, byte);
        if constexpr (QS)
            oq[c] = (uint32_t)(row * p.ldq + min<int64_t>(byte, (p.J - j0) * ES - 16));
        else
            oq[c] = (uint32_t)(min<int64_t>(row, p.J - j0 - 1) * p.ldq + byte);
    }
    const char *Pt = PS ? P + i0 * ES : P + i0 * p.ldp;
    const char *Qt = QS ? Q + j0 * ES : Q + j0 * p.ldq;
    const int64_t dp = PS ? KR * p.ldp : STEP, dq = QS ? KR * p.ldq : STEP;

    // Load c of a step: CP for P's tile, then CQ for Q's.
    constexpr int LOADS = CP + CQ;
    const int whole = (int)(R / KR);  // steps without an end of r in them
    auto load = [&](int s, int buf, int c, bool main = false) {
        const bool isp = c < CP;
        const int k = isp ? c : c - CP;
        const char *src = isp ? Pt + s * dp : Qt + s * dq;
        const uint32_t to = lds0 + buf * BUF + wave * 1024 + (isp ? 0 : TP::BYTES) + k * NTH * 16;
        uint32_t o = isp ? op[k < CP ? k : 0] : oq[k < CQ ? k : 0];
        if (main || s < whole) {
            load_lds(src, o, to);
        } else {
            const int left = (int)(R - (int64_t)s * KR);
            int row, byte;
            if (isp)
                TP::place(tid + k * NTH, row, byte);
            else
                TQ::place(tid + k * NTH, row, byte);
            asm volatile("" : "+v"(o));  // widened here, not in registers kept for it
            const char *zero = reinterpret_cast<const char *>(&zero_chunk);
            load_lds(((isp ? PS : QS) ? row < left : byte < left * ES) ? src + o : zero, to);
        }
    };
    auto stage = [&](int s, int buf) {
#pragma unroll
        for (int c = 0; c < LOADS; ++c) load(s, buf, c);
    };

    // fp8: the scales of a step, read one step ahead
    float sx[NI], sw = 1.0f;
    int sxo[NI];
    const int64_t nb = (p.J + 127) / 128;
    const float *swp = nullptr;
    if constexpr (ET == F8) {
#pragma unroll
        for (int a = 0; a < NI; ++a)
            sxo[a] = (int)min<int64_t>(wi * (BI / WI) + a * 16 + (lane & 15), i1 - i0 - 1);
        if constexpr (SCALE == BAKRON_SCALE_BLOCK)
            swp = p.sq + ((int64_t)g * ((p.R + KR - 1) / KR) + t.s0) * nb + min<int64_t>((j0 + wj * (BJ / WJ)) / 128, nb - 1);
    }
    auto scales = [&](int s) {
        if constexpr (ET == F8) {
#pragma unroll
            for (int a = 0; a < NI; ++a) sx[a] = (p.sp + (t.s0 + s) * p.rows + i0)[sxo[a]];
            if constexpr (SCALE == BAKRON_SCALE_BLOCK) sw = swp[s * nb];
        }
    };

    floatx4 acc[NI][NJ];
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int b = 0; b < NJ; ++b) acc[a][b] = floatx4{0, 0, 0, 0};

    // Within a step the LDS reads run ahead of the products by one part, over the end
    // of the step too: the barrier that hands over a buffer stands before the last
    // part's products, whose operands are in registers by then.
    const int ip = wi * (BI / WI), jq = wj * (BJ / WJ);
    if (steps > 0) {
        if constexpr (ET == F8) {
            stage(0, 0);
            scales(0);
            stage_wait();
            if (steps > 1)
#pragma unroll
                for (int c = 0; c < NI; ++c) load(1, 1, c);
            static_assert(LOADS >= NI && LOADS - NI <= NI * (NJ - 1), "every load has its product");
            // P's tiles stay in registers for the step; Q's are read one ahead.  The
            // sums of a product are added two products later.
            intx4 fp[NI][2], fq[2][2];
            float sc[NI], nsc[NI];
            floatx4 sum[3];
#pragma unroll
            for (int a = 0; a < NI; ++a) {
                sc[a] = SCALE == BAKRON_SCALE_BLOCK ? sx[a] * sw : sx[a];
#pragma unroll
                for (int h = 0; h < 2; ++h) fp[a][h] = TP::read(lds, ip + a * 16, h, lane);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) fq[0][h] = TQ::read(lds + TP::BYTES, jq, h, lane);
            auto step = [&](int s, bool main) {
                const char *lq = lds + (s & 1) * BUF + TP::BYTES;
                const char *np = lds + (~s & 1) * BUF, *nq = np + TP::BYTES;
                scales(main ? s + 1 : min(s + 1, steps - 1));
#pragma unroll
                for (int b = 0; b < NJ; ++b) {
                    const bool last = b == NJ - 1;
                    if (last) {
                        stage_wait();
#pragma unroll
                        for (int a = 0; a < NI; ++a) {
                            nsc[a] = SCALE == BAKRON_SCALE_BLOCK ? sx[a] * sw : sx[a];
                            asm volatile("" : "+v"(nsc[a]));  // taken before the next loads are under way
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        fq[~b & 1][h] = last ? TQ::read(nq, jq, h, lane) : TQ::read(lq, jq + (b + 1) * 16, h, lane);
#pragma unroll
                    for (int a = 0; a < NI; ++a) {
                        const int n = b * NI + a;
                        sum[n % 3] = mfma_f8(fq[b & 1][0], fq[b & 1][1], fp[a][0], fp[a][1]);
                        if (last)
#pragma unroll
                            for (int h = 0; h < 2; ++h) fp[a][h] = TP::read(np, ip + a * 16, h, lane);
                        if (n >= 2) {
                            const int m = n - 2;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[m % NI][m / NI][v] = fmaf(sc[m % NI], sum[m % 3][v], acc[m % NI][m / NI][v]);
                            asm volatile("" : "+v"(acc[m % NI][m / NI]));  // added here, not later
                        }
                        // the loads of a step, spread over the products that follow the barrier
                        if (last && (main || s + 2 < steps)) load(s + 2, s & 1, a, main);
                        if (n < LOADS - NI && (main || s + 1 < steps)) load(s + 1, ~s & 1, n + NI, main);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int m = NI * NJ - 2; m < NI * NJ; ++m)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[m % NI][m / NI][v] = fmaf(sc[m % NI], sum[m % 3][v], acc[m % NI][m / NI][v]);
#pragma unroll
                for (int a = 0; a < NI; ++a) sc[a] = nsc[a];
            };
            int s = 0;
            for (; s + 2 < whole; ++s) step(s, true);
            for (; s < steps; ++s) step(s, false);
        } else {
            // The two halves of a step each have their operands in registers when their
            // products begin: the second half's are read during the first, the next
            // step's first during the second.  The barrier between the halves says that
            // the step's buffer has been read, so the second half also issues the loads
            // of step s + NB, which have NB - 1 steps' time.
            constexpr int ALL = NI * NJ, READS = NI + NJ;
            static_assert(2 * READS <= ALL && ALL % LOADS == 0, "room between the products");
            intx4 fp[2][NI], fq[2][NJ];
            // operand i of half h of step s, in the order of use
            auto read = [&](int s, int h, int i) {
                const char *lp = lds + (s & (NB - 1)) * BUF;
                if (i == 0 || i > NI)
                    fq[h][i ? i - NI : 0] = TQ::read(lp + TP::BYTES, jq + (i ? i - NI : 0) * 16, h, lane);
                else
                    fp[h][i - 1] = TP::read(lp, ip + (i - 1) * 16, h, lane);
            };
            // main: the loads are there, and whole
            auto half = [&](int s, int h, bool main) {
#pragma unroll
                for (int n = 0; n < ALL; ++n) {
                    const int a = n % NI, b = n / NI;
                    if (n % 2 == 0 && n / 2 < READS) {
                        read(s + h, h ^ 1, n / 2);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    mfma_in_place<ET>(fq[h][b], fp[h][a], acc[a][b]);
                    if (h == 1 && n % (ALL / LOADS) == 1 && (main || s + NB < steps))
                        load(s + NB, s & (NB - 1), n / (ALL / LOADS), main);
                }
            };
            // of the `more` steps that were begun after the one that is waited for
            auto wait = [&](int more) {
                if (NB > 2 && more > 2)
                    stage_wait<3 * LOADS>();
                else if (NB > 2 && more == 2)
                    stage_wait<2 * LOADS>();
                else if (more == 1)
                    stage_wait<LOADS>();
                else
                    stage_wait();
            };
            const int begun = min(NB, steps);
            for (int s = 0; s < begun; ++s) stage(s, s);
            wait(begun - 1);
#pragma unroll
            for (int i = 0; i < READS; ++i) read(0, 0, i);
#pragma unroll
            for (int a = 0; a < NI; ++a)
#pragma unroll
                for (int b = 0; b < NJ; ++b) asm volatile("" : "+a"(acc[a][b]));
            settle();
            int s = 0;
            for (; s + NB < whole; ++s) {
                half(s, 0, true);
                stage_wait<(NB - 2) * LOADS>();
                half(s, 1, true);
            }
            for (; s < steps; ++s) {
                half(s, 0, false);
                wait(min(NB - 2, max(steps - 2 - s, 0)));
                half(s, 1, false);
            }
            settle();
#pragma unroll
            for (int a = 0; a < NI; ++a)
#pragma unroll
                for (int b = 0; b < NJ; ++b) asm volatile("" : "+a"(acc[a][b]));
        }
    }
    if (p.splits > 1) {
        store_part<NI, NJ>(p.part + t.nth * BI * BJ, acc, wave, lane);
        return;
    }
    // every wave is done with the operands' buffers, which now carry the results
    static_assert(512 * NI * NJ * WI * WJ <= NB * BUF, "the results of each wave");
    __syncthreads();
    store_tile<SCALE, NI, NJ, BI == 256>(p, acc, g, yoff, i0 + wi * (BI / WI), i1, j0 + wj * (BJ / WJ), lane,
                              lds + wave * 512 * NI * NJ);
}

template <int ET, int MODE, int SCALE, int NB, bool TAIL>
__global__ __launch_bounds__(256) void product_direct_kernel(ProductArgs p) {
    __shared__ __align__(1024) char lds[NB * 256 * STEP];
    direct_tile<ET, MODE, SCALE, 128, 128, 2, 2, NB>(p, blockIdx.x, TAIL, lds);
}

// 4 waves hold 128 x 128 accumulators each: a third less of LDS reads than 8 waves of
// 64 x 128 (bf16 8192 x 8192 x 8192 0.754 against 0.797 ms).  fp8 sums are added by
// vector instructions, which cannot use the registers that 4 waves need.
constexpr int large_waves(int et) { return et == F8 ? 8 : 4; }

// Large tiles; of 16-bit types, then their tail in small ones, which begins where the
// first CUs fall idle (bf16, 16384 rows by 8 groups of 11008 x 4096: 1.17 against 1.19
// ms as a second launch; 8192 x 4352 x 1024: 73 against 77 us).  fp8 tails gain from two
// workgroups on a CU instead, which the LDS of a large tile rules out (12000 rows by 16
// groups of 4096 x 2048: 133 us as a second launch, 141 here).
template <int ET, int MODE, int SCALE>
__global__ __launch_bounds__(64 * large_waves(ET)) void product_large_kernel(ProductArgs p) {
    constexpr int WI = large_waves(ET) / 2;
    __shared__ __align__(1024) char lds[2 * 512 * STEP];
    if (ET == F8 || blockIdx.x < p.large)
        direct_tile<ET, MODE, SCALE, 256, 256, WI, 2, 2>(p, blockIdx.x, false, lds);
    else if constexpr (ET != F8)
        direct_tile<ET, MODE, SCALE, 128, 128, WI, 2, 4>(p, blockIdx.x - p.large, true, lds);
}

// Few rows a group (decoding): the weights stream past once and bound the time, so
// they go straight from memory to registers.  A wave takes 16 rows of W and up to 16
// rows of X; the waves of a workgroup are wn sets of rows by wk parts of the
// reduction, which is dealt out in blocks of 128 bytes.  The parts' sums are added in
// a fixed order in LDS.  UNROLL blocks of both operands are loaded before the first is
// multiplied.  Loads that are not on whole dwords take three times as long (bf16, 4 rows
// by 4096 x 14337: 68 us, 28 at 14338 columns), so with ODD rows the dwords around
// a chunk are loaded and shifted (38 us).
__device__ __forceinline__ intx4 shifted(const intx4 &v, int next, uint32_t bytes) {
    intx4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = (int)__builtin_amdgcn_alignbyte((uint32_t)(i < 3 ? v[i < 3 ? i + 1 : 3] : next), (uint32_t)v[i], bytes);
    return r;
}
// 16 bytes from src's dword on, and the dword of src's 16th byte: no byte outside dwords
// that hold some of the 16 is read.
__device__ __forceinline__ void load_around(const char *src, intx4 &v, int &next) {
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(src) & 3;
    __builtin_memcpy(&v, __builtin_assume_aligned(src - off, 4), 16);
    __builtin_memcpy(&next, __builtin_assume_aligned(src - off + (off ? 16 : 12), 4), 4);
}
template <int ET, int SCALE, bool ODD>
__global__ __launch_bounds__(1024) void product_few_kernel(ProductArgs p, int wn) {
    constexpr int ES = ET == F8 ? 1 : 2, KR = STEP / ES, EC = 16 / ES, UNROLL = 4;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6, wk = waves / wn, kpart = wave / wn;
    const int l = lane & 15, q = lane >> 4;
    report_offsets(p);
    int g, tj;
    int64_t i0, i1, nth;
    if (!find_rows<16>(p, blockIdx.x, false, g, i0, i1, tj, nth)) return;
    g = (int)uniform(g), tj = (int)uniform(tj);
    i0 = uniform(i0), i1 = uniform(i1);
    const int64_t j0 = (int64_t)tj * 16 * wn + wave % wn * 16;
    const int blocks = g == p.groups ? 0 : (int)((p.R + KR - 1) / KR);  // no group: zeros
    const char *w = p.Q + (g == p.groups ? 0 : g) * p.group_q + min<int64_t>(j0 + l, p.J - 1) * p.ldq;
    const int64_t row = min<int64_t>(i0 + l, i1 - 1);
    const char *x = p.P + row * p.ldp;
    const int64_t nb = (p.J + 127) / 128;
    const float *sw = nullptr;
    if constexpr (SCALE == BAKRON_SCALE_BLOCK) sw = p.sq + (int64_t)g * blocks * nb + min<int64_t>(j0 / 128, nb - 1);
    floatx4 acc = {0, 0, 0, 0};

    for (int b0 = kpart; b0 < blocks; b0 += UNROLL * wk) {
        intx4 fw[UNROLL][2], fx[UNROLL][2];
        int nw[UNROLL][2], nx[UNROLL][2];
        float sc[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int b = b0 + u * wk;
            const int64_t left = b < blocks ? p.R - (int64_t)b * KR : 0;  // of r
            const int64_t at = (int64_t)b * STEP + q * 16;
            if (left >= KR) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (ODD) {
                        load_around(w + at + 64 * h, fw[u][h], nw[u][h]);
                        load_around(x + at + 64 * h, fx[u][h], nx[u][h]);
                    } else {
                        __builtin_memcpy(&fw[u][h], w + at + 64 * h, 16);
                        __builtin_memcpy(&fx[u][h], x + at + 64 * h, 16);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    nw[u][h] = nx[u][h] = 0;
                    fw[u][h] = chunk<ES>(w + at + 64 * h, left - (4 * h + q) * EC);
                    fx[u][h] = chunk<ES>(x + at + 64 * h, left - (4 * h + q) * EC);
                }
            }
            if constexpr (ET == F8) {
                sc[u] = left > 0 ? p.sp[b * p.rows + row] : 0.0f;
                if constexpr (SCALE == BAKRON_SCALE_BLOCK)
                    if (left > 0) sc[u] *= sw[b * nb];
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if constexpr (ODD) {
                const bool shift = b0 + u * wk < p.R / KR;
                const uint32_t bw = shift ? (uint32_t)reinterpret_cast<uintptr_t>(w) & 3 : 0;
                const uint32_t bx = shift ? (uint32_t)reinterpret_cast<uintptr_t>(x) & 3 : 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    fw[u][h] = shifted(fw[u][h], nw[u][h], bw);
                    fx[u][h] = shifted(fx[u][h], nx[u][h], bx);
                }
            }
            if constexpr (ET == F8) {
                const floatx4 s = mfma_f8(fw[u][0], fw[u][1], fx[u][0], fx[u][1]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[v] = fmaf(sc[u], s[v], acc[v]);
            } else {
                acc = mfma<ET>(fw[u][0], fx[u][0], acc);
                acc = mfma<ET>(fw[u][1], fx[u][1], acc);
            }
        }
    }
    floatx4 *part = reinterpret_cast<floatx4 *>(lds);
    if (wk > 1) {
        part[wave * 64 + lane] = acc;
        __syncthreads();
        if (kpart > 0) return;
        for (int k = 1; k < wk; ++k) acc += part[(wave + k * wn) * 64 + lane];
    }
    const int64_t j = j0 + 4 * q, i = i0 + l;
    if (i >= i1) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (j + v >= p.J) break;
        float y = acc[v];
        if constexpr (SCALE == BAKRON_SCALE_ROW) y = g == p.groups ? 0.0f : y * p.sq[g * p.J + j + v];
        const int64_t at = i * p.ldy + j + v;
        if (p.ytype == BAKRON_T_F32)
            store1<BAKRON_T_F32>(p.Y, at, y);
        else if (p.ytype == BAKRON_T_BF16)
            store1<BAKRON_T_BF16>(p.Y, at, y);
        else
            store1<BAKRON_T_F16>(p.Y, at, y);
    }
}

constexpr int64_t MAX_DIM = int64_t(1) << 24;
constexpr int32_t MAX_GROUPS = 4096;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int MODE, int BI, int BJ>
unsigned grid_of(ProductArgs &p) {
    p.tiles_j = (int)((p.J + BJ - 1) / BJ);
    p.tiles_i = (int)((p.I + BI - 1) / BI);
    if (MODE == GRAD_W) return (unsigned)((int64_t)p.groups * p.tiles_i * p.tiles_j);
    p.slots = (int)row_tiles(BI, p.rows, p.groups, p.offsets != nullptr);
    return (unsigned)((int64_t)p.slots * p.tiles_j);
}

// Tiles of b x b that a launch has, about: a group's last tile is half full on average,
// and the host does not know the sizes.
int64_t count_tiles(int mode, int64_t b, int64_t rows, int64_t I, int64_t J, int groups, bool grouped) {
    const int64_t tj = (J + b - 1) / b;
    if (mode == GRAD_W) return groups * ((I + b - 1) / b) * tj;
    return ((rows + b - 1) / b + (grouped ? groups / 2 : 0)) * tj;
}

// Which tile.  256 x 256 tiles need 128 KB of LDS, so a CU holds one; they move half
// the operand bytes of 128 x 128 tiles per product and are faster where they fill the
// chip (bf16 8192 x 8192 x 8192: 0.75 against 0.94 ms).  A launch of few tiles leaves
// CUs idle (fp8 2048 x 4096 x 4096: 51 against 41 us), and every group ends in a
// partial tile.  So: the rounds that each takes on 256 CUs (two small tiles fit on a
// CU), a round of large ones taking 1.5 times as long as one of small ones, or of a
// tail in small ones.
bool large_tiles(int mode, int64_t rows, int64_t I, int64_t J, int groups, bool grouped) {
    const int64_t big = count_tiles(mode, 256, rows, I, J, groups, grouped);
    const int64_t small = count_tiles(mode, 128, rows, I, J, groups, grouped);
    const int64_t whole = without_tail(big);
    return (whole + 255) / 256 * 3 + (whole < big ? 2 : 0) <= (small + 511) / 512 * 2;
}

// Into how many parts the reduction is split where small tiles are few: a step of a
// lone workgroup takes about 0.8 us, its loads' latency, whatever else is idle.  The
// second launch that adds the parts costs about 3 us, and a part of a tile, 64 KB out
// and in again, about 0.03 us (fp8 128 x 4096 x 4096, 32 tiles of 32 steps: 32 us
// whole, 22, 18.5 and 20 us in 2, 4 and 8 parts).
int choose_splits(int mode, int64_t rows, int64_t I, int64_t J, int64_t steps, int groups, bool grouped) {
    if (large_tiles(mode, rows, I, J, groups, grouped)) return 1;
    const int64_t tiles = count_tiles(mode, 128, rows, I, J, groups, grouped);
    const int64_t most = mode == GRAD_W ? tiles : row_tiles(128, rows, groups, grouped) * ((J + 127) / 128);
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 16 && s * 2 <= steps; s *= 2) {
        if (s > 1 && most * s > 4096) break;  // 256 MB of parts
        const double rounds = (double)((tiles * s + 511) / 512);
        const double t = (double)((steps + s - 1) / s) * 0.8 * rounds + (s > 1 ? 3.0 + tiles * s * 0.03 : 0.0);
        if (t < least * 0.95) least = t, best = s;
    }
    return best;
}

// Steps of the reduction; by group for the gradient of W.
int64_t steps_of(int mode, int es, int64_t rows, int64_t R, int groups) {
    return mode == GRAD_W ? (rows / groups * 2 + STEP - 1) / STEP : (R * es + STEP - 1) / STEP;
}

// Whether the rows are so few that the weights' one pass is the time: see
// product_few_kernel.  At one row a group it reads 5.0 TB/s where 128 x 128 tiles read
// 3.9 (64 rows, 64 groups of 2048 x 1024: 32 against 40 us); from 8 rows a group on the
// tiles are faster (57 against 67 us).
bool few_rows(int64_t rows, int groups, bool grouped) { return grouped ? rows <= 4 * groups : rows <= 16; }

// Bytes of the parts' sums.
size_t parts_size(int mode, int es, int64_t rows, int64_t I, int64_t J, int64_t R, int groups, bool grouped) {
    if (mode == FWD && few_rows(rows, groups, grouped)) return 0;
    const int s = choose_splits(mode, rows, I, J, steps_of(mode, es, rows, R, groups), groups, grouped);
    if (s == 1) return 0;
    const int64_t tj = (J + 127) / 128;
    const int64_t tiles = mode == GRAD_W ? groups * ((I + 127) / 128) * tj : row_tiles(128, rows, groups, grouped) * tj;
    return (size_t)(tiles * s) * 128 * 128 * sizeof(float);
}

// The parts of the reduction, wk, and the sets of rows of W, wn, of product_few_kernel's
// workgroups.  About 4096 waves, 16 a CU, keep enough loads under way: as many parts of
// the reduction as that takes, or sets of rows of W where one part does.
void few_waves(int es, int64_t rows, int64_t J, int64_t R, int groups, bool grouped, int &wn, int &wk) {
    const int64_t blocks = (R * es + STEP - 1) / STEP;
    const int64_t slots = grouped ? std::min<int64_t>(groups, rows) : (rows + 15) / 16;
    const int64_t sets = slots * ((J + 15) / 16);
    wk = 1;
    while (wk < 16 && wk * 2 * sets <= 4096 && wk * 2 <= blocks) wk *= 2;
    wn = wk >= 4 ? 1 : 4 / wk;
}

// Threads of the largest launch of a product, whichever form its operands' alignment
// calls for; rows after the last group's count too.  Split reductions are of few tiles.
int64_t launch_threads(int mode, int es, int64_t rows, int64_t I, int64_t J, int64_t R, int groups, bool grouped) {
    if (mode == FWD && few_rows(rows, groups, grouped)) {
        int wn, wk;
        few_waves(es, rows, J, R, groups, grouped, wn, wk);
        return row_tiles(16, rows, groups, grouped) * ((J + 16 * wn - 1) / (16 * wn)) * 64 * wn * wk;
    }
    auto tiles = [&](int64_t b) {
        return (mode == GRAD_W ? groups * ((I + b - 1) / b) : row_tiles(b, rows, groups, grouped)) * ((J + b - 1) / b);
    };
    return std::max(tiles(128) * 256, (tiles(256) + 7 + TAIL_MOST) * 512);
}

template <int ET, int SCALE>
void launch_few(ProductArgs &p, hipStream_t s) {
    int wn, wk;
    few_waves(ET == F8 ? 1 : 2, p.rows, p.J, p.R, p.groups, p.offsets != nullptr, wn, wk);
    p.tiles_j = (int)((p.J + 16 * wn - 1) / (16 * wn));
    p.slots = (int)row_tiles(16, p.rows, p.groups, p.offsets != nullptr);
    const int64_t grid = (int64_t)p.slots * p.tiles_j;
    const unsigned part = wk > 1 ? wn * wk * 1024 : 0;
    if (aligned(p.P, 4) && aligned(p.Q, 4) && p.ldp % 4 == 0 && p.ldq % 4 == 0)
        hipLaunchKernelGGL((product_few_kernel<ET, SCALE, false>), dim3((unsigned)grid), dim3(64 * wn * wk), part, s, p, wn);
    else
        hipLaunchKernelGGL((product_few_kernel<ET, SCALE, true>), dim3((unsigned)grid), dim3(64 * wn * wk), part, s, p, wn);
}

template <int ET, int MODE, int SCALE>
void launch(ProductArgs &p, hipStream_t s) {
    if constexpr (MODE == FWD)
        if (few_rows(p.rows, p.groups, p.offsets != nullptr)) return launch_few<ET, SCALE>(p, s);
    constexpr int ES = ET == F8 ? 1 : 2;
    // whole 16-byte chunks everywhere, and offsets inside a tile in 32 bits
    bool direct = aligned(p.P, 16) && aligned(p.Q, 16) && p.ldp % 16 == 0 && p.ldq % 16 == 0 &&
                  p.group_q % 16 == 0 && p.ldp < (1 << 22) && p.ldq < (1 << 22);
    direct = direct && (MODE == GRAD_W ? p.I * ES % 16 == 0 : p.R * ES % 16 == 0);
    direct = direct && (MODE == FWD || p.J * ES % 16 == 0);
    p.splits = 1;
    int splits = 1;
    if (p.part) {
        splits = choose_splits(MODE, p.rows, p.I, p.J, steps_of(MODE, ES, p.rows, p.R, p.groups), p.groups, p.offsets != nullptr);
    }
    if (direct && large_tiles(MODE, p.rows, p.I, p.J, p.groups, p.offsets != nullptr)) {
        const unsigned grid = grid_of<MODE, 256, 256>(p);
        // With groups of rows only the device knows how many tiles there are.
        p.tail = MODE != GRAD_W && p.offsets ? grid > 256 : without_tail(grid) < grid;
        p.large = (grid + 7) & ~7u;  // the tail's first workgroup goes to XCD 0
        hipLaunchKernelGGL((product_large_kernel<ET, MODE, SCALE>), dim3(p.large + (p.tail && ET != F8 ? TAIL_MOST : 0)),
                           dim3(64 * large_waves(ET)), 0, s, p);
        if constexpr (ET == F8)
            if (p.tail)
                hipLaunchKernelGGL((product_direct_kernel<ET, MODE, SCALE, 2, true>), dim3(TAIL_MOST), dim3(256), 0, s, p);
        return;
    }
    const unsigned grid = grid_of<MODE, 128, 128>(p);
    p.splits = splits;
    if (direct) {
        // 4 buffers where a CU gets one workgroup, as in the tail: loads have 3 steps' time
        // (gradients of 8192 rows by 16 groups of 4096 x 2048: 344 against 353 us, of 1003
        // by 24 of 1000 x 520: 31.4 against 33.5).  In the fp8 form the compiler's own
        // waits for the scales would wait for these loads too.
        constexpr int NB = ET == F8 ? 2 : 4;
        if (grid * splits <= 256)
            hipLaunchKernelGGL((product_direct_kernel<ET, MODE, SCALE, NB, false>), dim3(grid * splits), dim3(256), 0,
                               s, p);
        else
            hipLaunchKernelGGL((product_direct_kernel<ET, MODE, SCALE, 2, false>), dim3(grid * splits), dim3(256), 0,
                               s, p);
    } else {
        hipLaunchKernelGGL((product_kernel<ET, MODE, SCALE, 128, 128, 2, 2>), dim3(grid * splits), dim3(256), 0, s, p);
    }
    if (splits > 1) {
        hipLaunchKernelGGL((product_join_kernel<MODE, SCALE, STEP / ES>), dim3(grid * PIECES), dim3(64), 0, s, p, splits);
    }
}


bool sizes_ok(int64_t rows, int64_t N, int64_t K, int32_t groups) {
    return rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM && groups >= 1 &&
           groups <= MAX_GROUPS;
}

// Limits that keep every index in range: no size over 2^24, no more than 2^31
// workgroups of the smallest tiles, no launch of more threads than there can be.
int32_t check_sizes(int mode, int es, int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets) {
    BK_REQUIRE(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM,
               "bad sizes rows=%lld N=%lld K=%lld", (long long)rows, (long long)N, (long long)K);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    BK_REQUIRE(offsets || groups == 1, "offsets must be non-NULL for %d groups", groups);
    const int64_t I = mode == GRAD_W ? N : rows, J = mode == FWD ? N : K, R = mode == FWD ? K : mode == GRAD_X ? N : 0;
    BK_REQUIRE((rows / 16 + 1 + groups + 1) * (N / 16 + 1) < (int64_t(1) << 31) &&
                   (rows / 16 + 1 + groups + 1) * (K / 16 + 1) < (int64_t(1) << 31) &&
                   (int64_t)groups * (N / 64 + 1) * (K / 64 + 1) < (int64_t(1) << 31) &&
                   launch_threads(mode, es, rows, I, J, R, groups, offsets != nullptr) <= LAUNCH_THREADS,
               "too many tiles: rows=%lld N=%lld K=%lld groups=%d", (long long)rows, (long long)N,
               (long long)K, groups);
    return BAKRON_OK;
}

// `count` rows of stride `ld`: addresses stay below 2^56
int32_t check_ld(const char *name, int64_t ld, int64_t width, int64_t count) {
    BK_REQUIRE(ld >= width && ld <= MAX_LD && count <= (int64_t(1) << 54) / ld,
               "bad row stride %s=%lld for %lld rows of %lld", name, (long long)ld, (long long)count,
               (long long)width);
    return BAKRON_OK;
}

// The parts' sums, if the launch will have any.
int32_t take_parts(ProductArgs &p, int mode, int es, void *ws, size_t ws_bytes) {
    const size_t need = parts_size(mode, es, p.rows, p.I, p.J, p.R, p.groups, p.offsets != nullptr);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) {
        set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, ws_bytes);
        return BAKRON_ERR_WORKSPACE;
    }
    p.part = need ? static_cast<float *>(ws) : nullptr;
    return BAKRON_OK;
}

int32_t check_type16(int32_t type) {
    BK_REQUIRE(type == BAKRON_T_BF16 || type == BAKRON_T_F16, "type must be bf16 or fp16, not %d", type);
    return BAKRON_OK;
}

int32_t check_out(const void *Y, int32_t ytype, int32_t type) {
    BK_REQUIRE(ytype == type || ytype == BAKRON_T_F32, "the output's type must be the inputs' or fp32, not %d",
               ytype);
    BK_REQUIRE(aligned(Y, ytype == BAKRON_T_F32 ? 4 : 2), "the output is misaligned for its type");
    return BAKRON_OK;
}

int vector_rows(const void *Y, int32_t ytype, int64_t ld) {
    return ld * elem_size(ytype) % 16 == 0 && aligned(Y, 16);
}

}  // namespace
}  // namespace bakron

using namespace bakron;

#define BK_TRY(expr)                     \
    do {                                 \
        int32_t bk_r_ = (expr);          \
        if (bk_r_ != BAKRON_OK) return bk_r_; \
    } while (0)

extern "C" size_t bakron_fp8_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t groups) {
    if (!sizes_ok(rows, N, K, groups)) return 0;
    // one group may come with offsets or without
    return std::max(parts_size(FWD, 1, rows, rows, N, K, groups, true),
                    groups == 1 ? parts_size(FWD, 1, rows, rows, N, K, 1, false) : 0);
}

extern "C" size_t bakron_grouped_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t groups) {
    if (!sizes_ok(rows, N, K, groups)) return 0;
    size_t most = 0;
    for (bool grouped : {true, false}) {
        if (!grouped && groups != 1) continue;
        most = std::max({most, parts_size(FWD, 2, rows, rows, N, K, groups, grouped),
                         parts_size(GRAD_X, 2, rows, rows, K, N, groups, grouped),
                         parts_size(GRAD_W, 2, rows, N, K, 0, groups, grouped)});
    }
    return most;
}

extern "C" int32_t bakron_fp8_matmul(const uint8_t *X, int64_t ldx, const float *sx, const uint8_t *W,
                                     int64_t ldw, const float *sw, int32_t wscale, int64_t rows, int64_t N,
                                     int64_t K, int32_t groups, const int32_t *offsets, void *Y,
                                     int32_t ytype, int64_t ldy, int32_t *dev_status, void *ws,
                                     size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(X && sx && W && sw && Y, "X, sx, W, sw and Y must be non-NULL");
    BK_REQUIRE(wscale == BAKRON_SCALE_ROW || wscale == BAKRON_SCALE_BLOCK, "bad weight scale kind %d", wscale);
    BK_TRY(check_sizes(FWD, 1, rows, N, K, groups, offsets));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("ldy", ldy, N, rows));
    BK_TRY(check_type16(ytype));
    BK_TRY(check_out(Y, ytype, ytype));
    ProductArgs p = {};
    p.P = reinterpret_cast<const char *>(X), p.Q = reinterpret_cast<const char *>(W);
    p.Y = static_cast<char *>(Y);
    p.ldp = ldx, p.ldq = ldw, p.ldy = ldy, p.group_q = ldw * N;
    p.sp = sx, p.sq = sw;
    p.rows = p.I = rows, p.J = N, p.R = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = ytype;
    p.vec = vector_rows(Y, ytype, ldy);
    BK_TRY(take_parts(p, FWD, 1, ws, ws_bytes));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (wscale == BAKRON_SCALE_ROW)
        launch<F8, FWD, BAKRON_SCALE_ROW>(p, s);
    else
        launch<F8, FWD, BAKRON_SCALE_BLOCK>(p, s);
    BK_LAUNCH_CHECK("the fp8 product");
    return BAKRON_OK;
}

extern "C" int32_t bakron_grouped_matmul(const void *X, int32_t type, int64_t ldx, const void *W, int64_t ldw,
                                         int64_t rows, int64_t N, int64_t K, int32_t groups,
                                         const int32_t *offsets, void *Y, int32_t ytype, int64_t ldy,
                                         int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(X && W && Y, "X, W and Y must be non-NULL");
    BK_TRY(check_type16(type));
    BK_TRY(check_sizes(FWD, 2, rows, N, K, groups, offsets));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("ldy", ldy, N, rows));
    BK_TRY(check_out(Y, ytype, type));
    BK_REQUIRE(aligned(X, 2) && aligned(W, 2), "X or W is misaligned for its type");
    ProductArgs p = {};
    p.P = static_cast<const char *>(X), p.Q = static_cast<const char *>(W), p.Y = static_cast<char *>(Y);
    p.ldp = 2 * ldx, p.ldq = 2 * ldw, p.ldy = ldy, p.group_q = 2 * ldw * N;
    p.rows = p.I = rows, p.J = N, p.R = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = ytype;
    p.vec = vector_rows(Y, ytype, ldy);
    BK_TRY(take_parts(p, FWD, 2, ws, ws_bytes));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == BAKRON_T_BF16)
        launch<BAKRON_T_BF16, FWD, SCALE_NONE>(p, s);
    else
        launch<BAKRON_T_F16, FWD, SCALE_NONE>(p, s);
    BK_LAUNCH_CHECK("the grouped product");
    return BAKRON_OK;
}

extern "C" int32_t bakron_grouped_matmul_grad_x(const void *dY, int32_t type, int64_t lddy, const void *W,
                                                int64_t ldw, int64_t rows, int64_t N, int64_t K,
                                                int32_t groups, const int32_t *offsets, void *dX,
                                                int32_t dxtype, int64_t lddx, int32_t *dev_status,
                                                void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(dY && W && dX, "dY, W and dX must be non-NULL");
    BK_TRY(check_type16(type));
    BK_TRY(check_sizes(GRAD_X, 2, rows, N, K, groups, offsets));
    BK_TRY(check_ld("lddy", lddy, N, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("lddx", lddx, K, rows));
    BK_TRY(check_out(dX, dxtype, type));
    BK_REQUIRE(aligned(dY, 2) && aligned(W, 2), "dY or W is misaligned for its type");
    ProductArgs p = {};
    p.P = static_cast<const char *>(dY), p.Q = static_cast<const char *>(W), p.Y = static_cast<char *>(dX);
    p.ldp = 2 * lddy, p.ldq = 2 * ldw, p.ldy = lddx, p.group_q = 2 * ldw * N;
    p.rows = p.I = rows, p.J = K, p.R = N;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = dxtype;
    p.vec = vector_rows(dX, dxtype, lddx);
    BK_TRY(take_parts(p, GRAD_X, 2, ws, ws_bytes));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == BAKRON_T_BF16)
        launch<BAKRON_T_BF16, GRAD_X, SCALE_NONE>(p, s);
    else
        launch<BAKRON_T_F16, GRAD_X, SCALE_NONE>(p, s);
    BK_LAUNCH_CHECK("the grouped product's gradient");
    return BAKRON_OK;
}

extern "C" int32_t bakron_grouped_matmul_grad_w(const void *dY, int32_t type, int64_t lddy, const void *X,
                                                int64_t ldx, int64_t rows, int64_t N, int64_t K,
                                                int32_t groups, const int32_t *offsets, void *dW,
                                                int32_t dwtype, int64_t lddw, int32_t *dev_status,
                                                void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(dY && X && dW, "dY, X and dW must be non-NULL");
    BK_TRY(check_type16(type));
    BK_TRY(check_sizes(GRAD_W, 2, rows, N, K, groups, offsets));
    BK_TRY(check_ld("lddy", lddy, N, rows));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("lddw", lddw, K, groups * N));
    BK_TRY(check_out(dW, dwtype, type));
    BK_REQUIRE(aligned(dY, 2) && aligned(X, 2), "dY or X is misaligned for its type");
    ProductArgs p = {};
    p.P = static_cast<const char *>(dY), p.Q = static_cast<const char *>(X), p.Y = static_cast<char *>(dW);
    p.ldp = 2 * lddy, p.ldq = 2 * ldx, p.ldy = lddw, p.group_y = lddw * N;
    p.rows = rows, p.I = N, p.J = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = dwtype;
    p.vec = vector_rows(dW, dwtype, lddw);
    BK_TRY(take_parts(p, GRAD_W, 2, ws, ws_bytes));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == BAKRON_T_BF16)
        launch<BAKRON_T_BF16, GRAD_W, SCALE_NONE>(p, s);
    else
        launch<BAKRON_T_F16, GRAD_W, SCALE_NONE>(p, s);
    BK_LAUNCH_CHECK("the grouped product's gradient");
    return BAKRON_OK;
}
