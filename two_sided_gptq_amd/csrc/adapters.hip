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
// outer_kernel sums over a group's places.  In between P and U are kept in 32 bits, and go into
// the matrix cores as a sum of bf16 numbers, so that neither fp16's range nor bf16's 8 bits limit
// what lies between two products.  For results in 16 bits they are two numbers, hi + lo: what
// that loses, 2^-16 of a value, is far below half a step of the result (2^-11 in fp16).  For
// results in fp32 they are fp32 numbers, which three bf16 parts of 8 bits hold exactly.  The
// products of every part are exact in fp32 sums.
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
constexpr int MAX_SPLITS = 8;  // workgroups that share a tile's K

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
    uint32_t hi = f32_to_bf16(x);
    if ((hi & 0x7fff) == 0x7f80) hi = __float_as_uint(x) >> 16;  // rounded up to infinity: the largest below
    const float h = __uint_as_float(hi << 16);
    const uint32_t lo = __builtin_isfinite(h) ? f32_to_bf16(x - h) : 0;
    return hi << 16 | lo;
}
// Parts of the numbers between the products, by the type of the result.
constexpr int parts_of(int otype) { return otype == BAKRON_T_F32 ? 3 : 2; }
template <int PARTS>
__device__ __forceinline__ uint32_t pack(float x) {
    return PARTS == 2 ? pack_parts(x) : __float_as_uint(x);
}
// 8 packed numbers as the operands' fragments, one of each part.  Three: an fp32 number's upper
// 8 bits, those of what that leaves, and the rest, which has 8 at most.
template <int PARTS>
__device__ __forceinline__ void unpack_parts(const uint32_t *x, uintx4 (&part)[PARTS]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a = x[2 * j], b = x[2 * j + 1];
        if constexpr (PARTS == 2) {
            part[0][j] = __builtin_amdgcn_perm(b, a, 0x07060302);
            part[1][j] = __builtin_amdgcn_perm(b, a, 0x05040100);
        } else {
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                part[p][j] = __builtin_amdgcn_perm(b, a, 0x07060302);
                a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xffff0000u));
                b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xffff0000u));
            }
        }
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

// What lanes of a wave pass each other through LDS stays in the program's order; the hardware keeps
// it within a wave, so nothing is waited for.
__device__ __forceinline__ void order_lanes() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }

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

// The slot-th tile of `high` places, counted group by group (rows of no group last).
// before: how many tiles of `small` places the groups before it have, where asked for.
// most > 0: slots of groups are dealt so that neighbouring tiles, which share a group's
// matrices, share an XCD's L2; slot becomes the tile's number.  Only tiles that exist are
// dealt, or the last XCDs would have none, and no more than `most`, for which the
// workspace is sized: offsets that fall can make more.  Wave uniform.
__device__ __forceinline__ Tile tile_of(const Groups &a, int high, int &slot, int most, int small = 0,
                                        int *before = nullptr) {
    const int lane = threadIdx.x & 63;
    int64_t p, z;
    auto tiles_of = [&](int g) {
        p = z = 0;
        if (g <= a.groups) rows_of_group(a.offsets, a.groups, a.rows, g, p, z);
        return ((int)(z - p) + high - 1) / high;
    };
    int mine = tiles_of(lane), upto = wave_scan(mine), sum = 0;
    if (most > 0) {
        int all = __builtin_amdgcn_readlane(upto, min(a.groups - 1, 63));
        if (a.groups > 64) {
            for (int base = 64; base < a.groups; base += 64)
                all += __builtin_amdgcn_readlane(wave_scan(base + lane < a.groups ? tiles_of(base + lane) : 0), 63);
            mine = tiles_of(lane);
        }
        all = min(all, most);
        if (slot < all) slot = (int)xcd_order(slot, all);
    }
    int left = slot;
    for (int base = 0;;) {
        const int fine = before ? ((int)(z - p) + small - 1) / small : 0, fine_upto = before ? wave_scan(fine) : 0;
        const uint64_t hit = __ballot(left < upto);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            Tile t;
            t.g = base + src;
            const int first = __builtin_amdgcn_readlane((int)p, src), end = __builtin_amdgcn_readlane((int)z, src);
            t.p0 = first + (left - __builtin_amdgcn_readlane(upto - mine, src)) * high;
            t.p1 = min(end, t.p0 + high);
            t.pad = 0;
            if (before) *before = sum + __builtin_amdgcn_readlane(fine_upto - fine, src);
            return t;
        }
        left -= __builtin_amdgcn_readlane(upto, 63);
        if (before) sum += __builtin_amdgcn_readlane(fine_upto, 63);
        base += 64;
        if (base > a.groups) return {-1, 0, 0, 0};
        mine = tiles_of(base + lane);
        upto = wave_scan(mine);
    }
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
    const char *x, *w;      // rows of K values; a group's matrix
    int64_t ldx, group_w;
    int K, strided;         // the matrix is rank x K (0) or K x rank (1)
    uint32_t *by_place;     // [16-place tile][16][ranks], or NULL
    uint32_t *by_rank;      // [16-place tile][ranks][16], or NULL
    int place_parts, rank_parts;  // what they are packed as
};
struct ShrinkArgs {
    Groups of;
    Shrink job[2];
    const float *scale;     // of a group, or NULL
    int rank, ranks;        // ranks: in whole 16s
    int high, slots;        // places of a tile, tiles
    int splits;             // workgroups that share K, without GRAD: sums are then left in parts
    int64_t part_words;     // of a part
    Tile *tiles;            // written by the first job, as are
    int32_t *rows;          // the rows of the tiles' places
};

// The least tile is for few rows: its workgroup streams K with as many waves as fit.
constexpr int shrink_waves(int mt, int rt) { return mt == 1 && rt == 1 ? 16 : 8; }
constexpr int SHRINK_STEP = 64;  // values of K
constexpr int shrink_lds(int mt, int rt) {
    const int through = 16 * SHRINK_STEP * 2, sums = mt * rt * 1024;
    return shrink_waves(mt, rt) * (through > sums ? through : sums);
}

// GRAD: matrices of either order.  64 places by 64 ranks take the registers of a whole CU, and read
// half as much from L2 as 32 by 64 or by twice 32 (gradients, 8192 rows, 4096 x 4096, rank 64:
// 52 us instead of 67, rank 128: 83 instead of 118).  Of the others, 32 places by 64 ranks needs 3
// registers more than 4 waves a SIMD leave, and puts them aside in scratch memory.
template <int T, int MT, int RT, bool GRAD>
__global__ __launch_bounds__(64 * shrink_waves(MT, RT), MT * RT > 8 ? 2 : 4) void shrink_kernel(ShrinkArgs a) {
    extern __shared__ __align__(16) float space[];
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    constexpr int waves = shrink_waves(MT, RT), KS = SHRINK_STEP, DEPTH = MT * RT == 1 ? 3 : MT * RT == 2 ? 2 : 1;
    constexpr int CH = KS / 8, PER = 64 / CH, NL = 16 / PER;  // chunks of a row; rows of a load, loads of 16 rows
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int parts = a.high / (16 * MT), r0 = blockIdx.y * RT * 16;
    // the parts of a tile lie 8 apart, on one XCD
    const int block = blockIdx.x, sub = (block >> 3) % parts * MT;
    int slot = (block >> 3) / parts * 8 + (block & 7);
    if (slot >= a.slots) return;
    const Shrink &job = a.job[GRAD ? blockIdx.z : 0];
    const int part = GRAD ? 0 : blockIdx.z, splits = GRAD ? 1 : a.splits;
    Tile t = tile_of(a.of, a.high, slot, a.slots);
    if (blockIdx.y == 0 && blockIdx.z == 0 && sub == 0) {
        if (threadIdx.x == 0) a.tiles[slot] = t;
        if ((int)threadIdx.x < a.high) a.rows[slot * a.high + threadIdx.x] = row_at(a.of, t.p0 + threadIdx.x, t.p1);
        report(a.of, t, block == 0);
    }
    t.p0 += sub * 16;
    if (t.g < 0 || t.g == a.of.groups || t.p0 >= t.p1) return;
    // Loads go by neighbouring lanes along a row, KS values of it: 16 lanes of a load that lie in
    // 16 rows, as the matrix cores want them, take 16 cycles for 256 bytes instead of 4 (64
    // rows, K = 16384: 31 against 13 us).  A step's 16 rows pass through LDS of the wave's own,
    // 16-byte chunk c of row r at place c ^ r.
    // Places past the tile and ranks past the last read a row that exists; their results
    // are not used.
    const int lr = lane / CH, lc = lane % CH;
    const char *m = job.w + 2 * t.g * job.group_w, *x[MT][NL];
    const bool strided = GRAD && job.strided, whole_ranks = a.rank % 8 == 0;
    const uint32_t wide = (uint32_t)job.K * 2, narrow = (uint32_t)a.rank * 2;
    // 16 ranks of a step.  rank x K: as the rows of X.  K x rank: a lane has one of the 64 rows.
    auto load_w = [&](int s, int j, uintx4(&gm)[NL]) {
        int from = r0 + j * 16;
        asm("" : "+s"(from));  // addresses are made anew: there are no registers for all of them
        if (!strided) {
#pragma unroll
            for (int h = 0; h < NL; ++h)
                gm[h] = load_whole(m + lc * 16 + (uint64_t)wide * (uint32_t)min(from + lr + h * PER, a.rank - 1), s * KS);
        } else {
#pragma unroll
            for (int h = 0; h < NL; ++h) {
                const char *row = m + (uint64_t)narrow * (uint32_t)(s * KS + lane);
                const int r = from + h * 8;
                gm[h] = whole_ranks ? load_whole(row, min(r, a.rank - 8)) : load_frag(row, r, a.rank - r);
            }
        }
    };
    auto load_w_tail = [&](int k, int j, uintx4(&gm)[NL]) {
#pragma unroll
        for (int h = 0; h < NL; ++h) {
            const int r = r0 + j * 16 + h * 8;
            if (!strided)
                gm[h] = load_frag(m + (uint64_t)wide * (uint32_t)min(r0 + j * 16 + lr + h * PER, a.rank - 1), k + lc * 8,
                                  job.K - k - lc * 8);
            else
                gm[h] = load_frag(m + (uint64_t)narrow * (uint32_t)min(k + lane, job.K - 1), r, k + lane < job.K ? a.rank - r : 0);
        }
    };
    floatx4 acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = floatx4{0, 0, 0, 0};
    // KS of K a step, DEPTH steps on their way.  Workgroups begin at different columns: rows of
    // a power of two in bytes would otherwise have all of them at the same memory channels.
    const int whole = job.K / KS, turned = whole ? (int)((int64_t)blockIdx.x * waves % whole) : 0;
    const int all = waves * splits, first = part * waves + w;  // waves that share K
    auto step = [&](int s) { return s + turned < whole ? s + turned : s + turned - whole; };
    uintx4 vx[DEPTH][MT][NL], vm[DEPTH][RT][NL];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (first + d * all < whole)
#pragma unroll
            for (int j = 0; j < RT; ++j) load_w(step(first + d * all), j, vm[d][j]);
    int row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        row[i] = row_at(a.of, t.p0 + i * 16 + l, t.p1);
#pragma unroll
        for (int h = 0; h < NL; ++h) x[i][h] = job.x + 2 * (max(__shfl(row[i], h * PER + lr), 0) * job.ldx + lc * 8);
    }
    auto load_x = [&](int s, int i, uintx4(&gx)[NL]) {
#pragma unroll
        for (int h = 0; h < NL; ++h) gx[h] = load_whole(x[i][h], s * KS);
    };
    char *own = reinterpret_cast<char *>(space) + w * (16 * KS * 2);
    auto through = [&](const uintx4(&v)[NL], uintx4(&f)[NL]) {
#pragma unroll
        for (int h = 0; h < NL; ++h) {
            const int r = h * PER + lr;
            *reinterpret_cast<uintx4 *>(own + r * (KS * 2) + (lc ^ (r & (CH - 1))) * 16) = v[h];
        }
        order_lanes();
#pragma unroll
        for (int h = 0; h < NL; ++h)
            f[h] = *reinterpret_cast<const uintx4 *>(own + l * (KS * 2) + ((h * 4 + q) ^ (l & (CH - 1))) * 16);
        order_lanes();
    };
    // K x rank: rows of 32 bytes, read with a transposing load: lane l of 16 gets rank l and 4
    // of K from each.
    auto through_strided = [&](const uintx4(&v)[NL], uintx4(&f)[NL]) {
        typedef short shortx4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) shortx4 *lds4;
#pragma unroll
        for (int h = 0; h < NL; ++h) *reinterpret_cast<uintx4 *>(own + lane * 32 + h * 16) = v[h];
        order_lanes();
#pragma unroll
        for (int h = 0; h < NL; ++h) {
            char *at = own + (h * 32 + q * 8 + (l >> 2)) * 32 + (l & 3) * 8;
            const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at));
            const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 4 * 32));
            __builtin_memcpy(&f[h], &lo, 8);
            __builtin_memcpy(reinterpret_cast<char *>(&f[h]) + 8, &hi, 8);
        }
        order_lanes();
    };
    // Registers take the loads of step `next` as soon as LDS has what they held.
    auto multiply = [&](uintx4(&gx)[MT][NL], uintx4(&gm)[RT][NL], int next) {
        uintx4 fx[MT][NL];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            through(gx[i], fx[i]);
            if (next < whole) load_x(step(next), i, gx[i]);
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            uintx4 fm[NL];
            if (strided)
                through_strided(gm[j], fm);
            else
                through(gm[j], fm);
            if (next < whole) load_w(step(next), j, gm[j]);
#pragma unroll
            for (int h = 0; h < NL; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][j] = mfma<T>(fx[i][h], fm[h], acc[i][j]);
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (first + d * all < whole)
#pragma unroll
            for (int i = 0; i < MT; ++i) load_x(step(first + d * all), i, vx[d][i]);
    for (int s = first; s < whole; s += DEPTH * all) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (s + d * all < whole) multiply(vx[d], vm[d], s + (d + DEPTH) * all);
    }
    if (whole * KS < job.K && first == whole % all) {
        const int k = whole * KS, left = job.K - k - lc * 8;
#pragma unroll
        for (int h = 0; h < NL; ++h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) vx[0][i][h] = load_frag(x[i][h], k, left);
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) load_w_tail(k, j, vm[0][j]);
        multiply(vx[0], vm[0], whole);
    }
    __syncthreads();
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
            const int64_t tile = (int64_t)slot * (a.high / 16) + sub + i;
            const int rank = r0 + j * 16 + l;
            uintx4 whole, packed;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool ok = __shfl(row[i], q * 4 + e) >= 0 && rank < a.rank;
                const float x = ok ? s[e] * scale : 0.0f;
                whole[e] = pack<3>(x), packed[e] = pack<2>(x);
            }
            if (job.by_rank)
                *reinterpret_cast<uintx4 *>(job.by_rank + (tile * a.ranks + rank) * 16 + q * 4) = job.rank_parts == 2 ? packed : whole;
            if (job.by_place) {
                const uintx4 v = job.place_parts == 2 && splits == 1 ? packed : whole;
#pragma unroll
                for (int e = 0; e < 4; ++e) job.by_place[part * a.part_words + (tile * 16 + q * 4 + e) * a.ranks + rank] = v[e];
            }
        }
}

// ---------------------------------------------------------------- expand

struct ExpandArgs {
    Groups of;
    const Tile *tiles;
    const int32_t *rows;    // of the tiles' places
    const uint32_t *p;      // [16-place tile][16][ranks]; with splits > 1 so many parts of sums in fp32
    int splits;
    int64_t part_words;
    const char *w;          // a group's matrix
    int64_t group_w;        // STRIDED: rank x N, else N x rank
    const char *base;       // may be out; NULL: 0
    char *out;
    int64_t ldb, ldo;
    int N, rank, ranks;
    int per_chunk;          // 2^16 / (rank / 8), rounded up: divides what is below 2^11
};

// The products of a matrix's fragment with every part of P's or U's.
template <int T, int PARTS>
__device__ __forceinline__ void add_products(const uintx4 &f, const uintx4 (&part)[PARTS], floatx4 &acc) {
    if constexpr (T == BAKRON_T_BF16) {
#pragma unroll
        for (int p = 0; p < PARTS; ++p) acc = mfma_bf16(f, part[p], acc);
    } else {
        uintx4 fh, fl;
        split_f16(f, fh, fl);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) acc = mfma_bf16(fh, part[p], acc);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) acc = mfma_bf16(fl, part[p], acc);
    }
}

// P of the tile's places, on its way from memory, 16 bytes a thread and turn; then to LDS,
// rows of `ranks` 4 words apart.
template <int MT, int RS, int PARTS>
struct StagedP {
    static constexpr int TURNS = (MT * RS + 1) / 2;
    uintx4 v[TURNS];
    __device__ __forceinline__ void load(const ExpandArgs &a, int64_t slot, int words) {
        const uint32_t *p = a.p + slot * MT * 16 * a.ranks;
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int i = k * 1024 + threadIdx.x * 4;
            if (i < words) v[k] = *reinterpret_cast<const uintx4 *>(p + i);
        }
        if (MT > 1 || a.splits == 1) return;
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int i = k * 1024 + threadIdx.x * 4;
            if (i >= words) break;
            floatx4 sum = __builtin_bit_cast(floatx4, v[k]);
#pragma unroll 1
            for (int m = 1; m < a.splits; ++m) sum += *reinterpret_cast<const floatx4 *>(p + m * a.part_words + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] = pack<PARTS>(sum[e]);
        }
    }
    __device__ __forceinline__ void store(const ExpandArgs &a, int words, uint32_t *lds) const {
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int i = k * 1024 + threadIdx.x * 4, r = i / a.ranks;
            if (i < words) *reinterpret_cast<uintx4 *>(lds + r * (a.ranks + 4) + (i - r * a.ranks)) = v[k];
        }
    }
};

template <int PARTS>
__device__ __forceinline__ void p_frags(const ExpandArgs &a, const uint32_t *lds, int place, int r, uintx4 (&part)[PARTS]) {
    uint32_t p[8] = {};
    if (r < a.ranks) __builtin_memcpy(p, __builtin_assume_aligned(lds + place * (a.ranks + 4) + r, 16), 32);
    unpack_parts(p, part);
}

constexpr int EXPAND_ROW = 68;  // floats between the rows of results in LDS

// D = W P^T with W's rows as the first operand: a lane then holds 4 of W's rows (columns of
// out) for one place.  A workgroup takes a tile's places and 256 columns, a wave 64 of
// them: W's part stays in registers, P in LDS.
//
// All that is in memory is read and written along rows by neighbouring lanes (see
// shrink_kernel), and passes through LDS of the wave's own to and from the lanes that the
// matrix cores want it in.  All loads are on their way before the first is waited for.
// Needs 256 columns and, where W is N x rank, ranks in whole 8s.
template <int T, int OT, int MT, int RS, bool STRIDED>
__device__ __forceinline__ void expand_whole(const ExpandArgs &a, const Tile &t, int64_t slot, int n0, uint32_t *lds, char *own) {
    constexpr int OS = OT == BAKRON_T_F32 ? 4 : 2, PARTS = parts_of(OT);
    constexpr int PER = RS == 1 ? 4 : 1;          // 16-row pieces of W that pass at a time
    constexpr int WL = RS == 1 ? 4 : 2 * RS / 2;  // loads of a pass
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
    const bool none = t.g == a.of.groups;
    const int count = t.p1 - t.p0;
    const int words = none ? 0 : (count + 15) / 16 * 16 * a.ranks;
    StagedP<MT, RS, PARTS> p;
    p.load(a, slot, words);
    int row[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int place = i * 16 + h * 8 + lr, r = a.rows[slot * (16 * MT) + place];
            row[i][h] = place < count ? r : -1;
        }
    const int chunks = a.rank / 8, some = 16 * PER * chunks;  // 16-byte pieces of a row, of a pass
    const char *wg = a.w + 2 * ((none ? 0 : t.g) * a.group_w);
    uintx4 raw_w[4 * RS];
    if constexpr (!STRIDED) {
        // W's 64 rows are one stretch of memory
        wg += 2 * (int64_t)n0 * a.rank;
#pragma unroll
        for (int c = 0; c < 4 / PER; ++c)
#pragma unroll
            for (int k = 0; k < WL; ++k)
                if (k * 64 + lane < some) raw_w[c * WL + k] = load_whole(wg, (int64_t)(c * some + k * 64 + lane) * 8);
    } else {
        // 64 columns of all ranks, 8 rows a load
        wg += 2 * (n0 + lc * 8);
#pragma unroll
        for (int k = 0; k < 4 * RS; ++k) {
            raw_w[k] = uintx4{0, 0, 0, 0};
            if (k * 8 < a.rank) {
                raw_w[k] = load_whole(wg, (int64_t)min(k * 8 + lr, a.rank - 1) * a.N);
                if (k * 8 + lr >= a.rank) raw_w[k] = uintx4{0, 0, 0, 0};
            }
        }
    }
    // places without a row read row 0 and write nothing
    Raw8<OT> base[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            base[i][h] = Raw8<OT>{};
            if (a.base) __builtin_memcpy(base[i][h].w, a.base + OS * (max(row[i][h], 0) * a.ldb + n0 + lc * 8), 8 * OS);
        }
    p.store(a, words, lds);
    __syncthreads();
    uintx4 f[4][RS];
    if constexpr (!STRIDED) {
#pragma unroll
        for (int c = 0; c < 4; c += PER) {
#pragma unroll
            for (int k = 0; k < WL; ++k) {
                const int i = k * 64 + lane, r = i * a.per_chunk >> 16;  // i / chunks
                if (i < some) *reinterpret_cast<uintx4 *>(own + (i + r) * 16) = raw_w[c / PER * WL + k];
            }
            order_lanes();
#pragma unroll
            for (int d = 0; d < PER; ++d)
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    f[c + d][s] = uintx4{0, 0, 0, 0};
                    if (s * 4 + q < chunks)
                        f[c + d][s] = *reinterpret_cast<const uintx4 *>(own + ((d * 16 + l) * (chunks + 1) + s * 4 + q) * 16);
                }
            order_lanes();
        }
    } else {
        // rows of 128 bytes, the 32 of 16 columns at place c ^ (row & 3), read with a transposing load
        typedef short shortx4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) shortx4 *lds4;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = k * 8 + lr;
                *reinterpret_cast<uintx4 *>(own + r * 128 + (((lc >> 1) ^ (r & 3)) * 32) + (lc & 1) * 16) = raw_w[s * 4 + k];
            }
            order_lanes();
            const int r = q * 8 + (l >> 2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                char *at = own + r * 128 + (c ^ (r & 3)) * 32 + (l & 3) * 8;
                const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at));
                const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 4 * 128));
                __builtin_memcpy(&f[c][s], &lo, 8);
                __builtin_memcpy(reinterpret_cast<char *>(&f[c][s]) + 8, &hi, 8);
            }
            order_lanes();
        }
    }
    float *results = reinterpret_cast<float *>(own);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if (i * 16 >= count) break;
        floatx4 acc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = floatx4{0, 0, 0, 0};
        if (!none) {
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                uintx4 part[PARTS];
                p_frags(a, lds, i * 16 + l, s * 32 + q * 8, part);
#pragma unroll
                for (int c = 0; c < 4; ++c) add_products<T>(f[c][s], part, acc[c]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) *reinterpret_cast<floatx4 *>(results + l * EXPAND_ROW + c * 16 + q * 4) = acc[c];
            order_lanes();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[8];
            unpack8<OT>(base[i][h].w, y);
            if (!none) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const floatx4 d = *reinterpret_cast<const floatx4 *>(results + (h * 8 + lr) * EXPAND_ROW + lc * 8 + e * 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[e * 4 + k] += d[k];
                }
            }
            if (row[i][h] >= 0) store8<OT>(a.out, row[i][h] * a.ldo + n0 + lc * 8, 8, y);
        }
        order_lanes();
    }
}

// The same for any N and rank: lanes read and write where the matrix cores have them.  The 64
// columns are dealt to the 4 products so that a lane's are two runs of 8: row m of product
// c is column 32 (c / 2) + 8 (m / 4) + 4 (c % 2) + m % 4.
template <int T, int OT, int MT, int RS, bool STRIDED>
__device__ __forceinline__ void expand_any(const ExpandArgs &a, const Tile &t, int64_t slot, int n0, uint32_t *lds) {
    constexpr int PARTS = parts_of(OT);
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const bool none = t.g == a.of.groups;
    const int count = t.p1 - t.p0, col = n0 + q * 8, left = a.N - col;
    uintx4 f[4][RS];
    const char *wg = a.w + 2 * ((none ? 0 : t.g) * a.group_w);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int n = min(n0 + (c >> 1) * 32 + (l >> 2) * 8 + (c & 1) * 4 + (l & 3), a.N - 1);
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            const int r = s * 32 + q * 8;
            if constexpr (!STRIDED) {
                f[c][s] = load_frag(wg, (int64_t)n * a.rank + r, a.rank - r);
            } else {
                f[c][s] = uintx4{0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (r + e < a.rank)
                        f[c][s][e / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(wg)[(int64_t)(r + e) * a.N + n] << (16 * (e & 1));
            }
        }
    }
    StagedP<MT, RS, PARTS> p;
    const int words = none ? 0 : (count + 15) / 16 * 16 * a.ranks;
    p.load(a, slot, words);
    p.store(a, words, lds);
    __syncthreads();
    for (int i = 0; i * 16 < count; ++i) {
        const int row = i * 16 + l < count ? a.rows[slot * (16 * MT) + i * 16 + l] : -1;
        float y[2][8] = {};
        if (a.base && row >= 0)
#pragma unroll
            for (int h = 0; h < 2; ++h) load8<OT>(a.base, row * a.ldb + col + 32 * h, left - 32 * h, y[h]);
        if (!none) {
            floatx4 acc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                uintx4 part[PARTS];
                p_frags(a, lds, i * 16 + l, s * 32 + q * 8, part);
#pragma unroll
                for (int c = 0; c < 4; ++c) add_products<T>(f[c][s], part, acc[c]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[c >> 1][(c & 1) * 4 + e] += acc[c][e];
        }
        if (row >= 0)
#pragma unroll
            for (int h = 0; h < 2; ++h) store8<OT>(a.out, row * a.ldo + col + 32 * h, left - 32 * h, y[h]);
    }
}

// LDS of a workgroup: P, and what passes through for each wave.
__host__ __device__ constexpr int expand_p_words(int mt, int ranks) { return 16 * mt * (ranks + 4); }
__host__ __device__ constexpr int expand_own_bytes(int rank) {
    // W as N x rank; as rank x N 4 KB, less than the results
    const int w = (rank <= 32 ? 64 : 16) * (rank / 8 + 1) * 16, results = 16 * EXPAND_ROW * 4;
    return w > results ? w : results;
}

template <int T, int OT, int MT, int RS, bool STRIDED>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs a) {
    extern __shared__ __align__(16) uint32_t lds[];
    const int blocks = (a.N + 255) / 256;
    const int64_t slot = blockIdx.x / blocks;
    const int first = (int)(blockIdx.x - slot * blocks) * 256, n0 = first + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64;
    const Tile t = a.tiles[slot];
    if (t.g < 0 || (t.g == a.of.groups && a.base == a.out)) return;
    if ((STRIDED || a.rank % 8 == 0) && first + 256 <= a.N)
        expand_whole<T, OT, MT, RS, STRIDED>(a, t, slot, n0, lds, reinterpret_cast<char *>(lds + expand_p_words(MT, a.ranks)) +
                                                            (threadIdx.x >> 6) * expand_own_bytes(a.rank));
    else
        expand_any<T, OT, MT, RS, STRIDED>(a, t, slot, n0, lds);
}

// ---------------------------------------------------------------- outer

// G_g^T Z_g over a group's places: dA (rank x K, Z = X, G = U) or dB (N x rank, Z = dY, G = P).
struct Outer {
    const char *z;
    int64_t ldz;
    int cols;               // K or N
    const uint32_t *g;      // by_rank
    char *out;
    int64_t group_o;        // elements
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
// A workgroup takes a unit's places, 128 columns and 16 RT ranks; its waves share the
// places, 32 at a time.  A lane reads 8 columns of 8 rows and turns them about with byte
// permutes: the matrix cores want 8 places of one column.  2 or 8 waves (gradients of 4000 rows
// by 64 groups, 4096 x 4096: 63 us with 2, 84 with 8).
template <int T, int WAVES, int RT, int PARTS, bool WHOLE>
__device__ __forceinline__ void outer_sum(const OuterArgs &a, const Outer &job, const Tile &t, int64_t sub, int c0, int r0,
                                          floatx4 (&acc)[8][RT]) {
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = c0 + l * 8, left = job.cols - col, count = t.p1 - t.p0;
    // the rows of the next 32 places, one a lane
    int next = row_at(a.of, t.p0 + w * 32 + (lane & 31), t.p1);
    for (int s = w * 32; s < count; s += WAVES * 32) {
        const int row = next;
        next = row_at(a.of, t.p0 + s + WAVES * 32 + (lane & 31), t.p1);
        uintx4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int r = __shfl(row, q * 8 + e);
            const int64_t at = max(r, 0) * job.ldz + col;
            if constexpr (WHOLE)
                v[e] = load_whole(job.z, at);
            else
                v[e] = load_frag(job.z, at, r >= 0 ? left : 0);
        }
        uint32_t g[RT][8];
        const int64_t tile = sub + s / 16 + (q >> 1);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int rank = r0 + r * 16 + l;
#pragma unroll
            for (int k = 0; k < 8; ++k) g[r][k] = 0;
            // past the unit's last 16-place tile there is none (nor where offsets fall)
            if (rank < a.ranks && tile >= 0 && tile < a.subs && s + (q & 2) * 8 < count)
                __builtin_memcpy(g[r], job.g + (tile * a.ranks + rank) * 16 + (q & 1) * 8, 32);
        }
        // places without a row: what was read from row 0 does not count
        if (WHOLE && __any(row < 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (__shfl(row, q * 8 + e) < 0) v[e] = uintx4{0, 0, 0, 0};
        }
        uintx4 part[RT][PARTS];
#pragma unroll
        for (int r = 0; r < RT; ++r) unpack_parts(g[r], part[r]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uintx4 f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __builtin_amdgcn_perm(v[2 * j + 1][c / 2], v[2 * j][c / 2], c & 1 ? 0x07060302 : 0x05040100);
#pragma unroll
            for (int r = 0; r < RT; ++r) add_products<T>(f, part[r], acc[c][r]);
        }
    }
}

template <int T, int WAVES, int RT, int PARTS>
__global__ __launch_bounds__(64 * WAVES) void outer_kernel(OuterArgs a) {
    // half of the waves' sums; then the results as rows of the output
    constexpr int HALF = WAVES / 2 * 8 * RT * 256, BY_RANK = 128 + 4, BY_COLUMN = 16 * RT + 4;
    constexpr int RESULTS = BY_RANK * 16 * RT > BY_COLUMN * 128 ? BY_RANK * 16 * RT : BY_COLUMN * 128;
    __shared__ __align__(16) float room[HALF > RESULTS ? HALF : RESULTS];
    floatx4 *space = reinterpret_cast<floatx4 *>(room);
    const Outer &job = a.job[blockIdx.z];
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wide = (max(a.job[0].cols, a.job[1].cols) + 127) / 128;
    const int unit = blockIdx.x / wide, c0 = ((int)blockIdx.x - unit * wide) * 128, r0 = blockIdx.y * RT * 16;
    if (c0 >= job.cols) return;
    Tile t;
    int before;
    int64_t p, z;
    if (a.chunk) {
        int at = unit;
        t = tile_of(a.of, a.chunk, at, 0, a.high, &before);
        if (t.g < 0 || t.g == a.of.groups) return;
        rows_of_group(a.of.offsets, a.of.groups, a.of.rows, t.g, p, z);
    } else {
        // all of group `unit`, also an empty one
        int sum = 0;
        for (int e = lane; e < unit; e += 64) {
            rows_of_group(a.of.offsets, a.of.groups, a.of.rows, e, p, z);
            sum += ((int)(z - p) + a.high - 1) / a.high;
        }
        before = __builtin_amdgcn_readlane(wave_scan(sum), 63);
        rows_of_group(a.of.offsets, a.of.groups, a.of.rows, unit, p, z);
        t = {unit, (int)p, (int)z, 0};
    }
    // shrink's 16-place tiles of this unit
    const int64_t sub = (int64_t)before * (a.high / 16) + (t.p0 - (int)p) / 16;
    floatx4 acc[8][RT];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[c][r] = floatx4{0, 0, 0, 0};
    if (c0 + 128 <= job.cols)
        outer_sum<T, WAVES, RT, PARTS, true>(a, job, t, sub, c0, r0, acc);
    else
        outer_sum<T, WAVES, RT, PARTS, false>(a, job, t, sub, c0, r0, acc);
    // the upper half of the waves to the lower, until one is left
#pragma unroll
    for (int half = WAVES / 2; half > 0; half >>= 1) {
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
    // lane: rank l, columns 8 (4 q + e) + c
    if (w == 0) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int rank = r * 16 + l, at = 8 * (4 * q + e) + c;
                    room[job.by_column ? at * BY_COLUMN + rank : rank * BY_RANK + at] = acc[c][r][e];
                }
    }
    __syncthreads();
    // the output's rows: of a rank, or of a column; a group's are contiguous
    const int length = job.by_column ? 16 * RT : 128, rows = job.by_column ? 128 : 16 * RT, pitch = job.by_column ? BY_COLUMN : BY_RANK;
    const int row0 = job.by_column ? c0 : r0, col1 = job.by_column ? r0 : c0;
    const int all_rows = job.by_column ? job.cols : a.rank, all_cols = job.by_column ? a.rank : job.cols;
    for (int i = threadIdx.x * 8; i < rows * length; i += 64 * WAVES * 8) {
        const int y = i / length, x = i - y * length, left = all_cols - (col1 + x);
        if (row0 + y >= all_rows || left <= 0) continue;
        const float *v = room + y * pitch + x;
        const int64_t at = (int64_t)(row0 + y) * all_cols + col1 + x;
        if (a.chunk)
            store8<BAKRON_T_F32>(reinterpret_cast<char *>(a.part), unit * a.part_size + job.part0 + at, left, v);
        else
            store_any(job.out, a.otype, t.g * job.group_o + at, left, v);
    }
}

// Adds a group's units, in order.  A thread takes 8 neighbours.
__global__ __launch_bounds__(256) void outer_join_kernel(OuterArgs a) {
    const Outer &job = a.job[blockIdx.z];
    const int g = blockIdx.y, lane = threadIdx.x & 63;
    int first = 0;
    int64_t p, z;
    for (int e = lane; e < g; e += 64) {
        rows_of_group(a.of.offsets, a.of.groups, a.of.rows, e, p, z);
        first += ((int)(z - p) + a.chunk - 1) / a.chunk;
    }
    first = __builtin_amdgcn_readlane(wave_scan(first), 63);
    rows_of_group(a.of.offsets, a.of.groups, a.of.rows, g, p, z);
    const int last = min(a.units, first + ((int)(z - p) + a.chunk - 1) / a.chunk);
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, left = (int64_t)a.rank * job.cols - i;
    if (left <= 0) return;
    float sum[8] = {};
    const char *from = reinterpret_cast<const char *>(a.part + job.part0 + i);
    for (int u0 = max(first, 0); u0 < last; u0 += 4) {
        float x[4][8] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (u0 + k < last) load8<BAKRON_T_F32>(from, (u0 + k) * a.part_size, left, x[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += x[k][e];
    }
    store_any(job.out, a.otype, g * job.group_o + i, (int)min<int64_t>(left, 8), sum);
}

// ---------------------------------------------------------------- layout and launches

// How a call is laid out; the same for workspace and launch.
struct Layout {
    int mt;                 // 16-place tiles of a tile of expand: 1 or 4
    int st, rt;             // 16-place tiles and 16-rank blocks of a workgroup of shrink
    int ranks, rs;          // ranks in whole 16s; 32-rank steps of expand
    int64_t slots;          // tiles of 16 mt places
    int splits;             // of K, in shrink
    int chunk;              // of the sums over places; 0: a group is one unit
    int64_t units;
    int outer_waves;        // waves that share a unit's places
};

Layout layout_of(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups, bool grad) {
    Layout y;
    y.ranks = (int)round_up(rank, 16);
    y.rs = rank <= 32 ? 1 : rank <= 64 ? 2 : rank <= 128 ? 4 : 8;
    y.mt = rows >= 64 * (int64_t)(groups + 1) && rows >= 1024 ? 4 : 1;
    y.slots = row_tiles(16 * y.mt, rows, groups, true);
    const int blocks = y.ranks / 16;
    // Gradients of 16 or 32 places take 32 ranks at most: with 64 and both orders of a matrix the
    // registers leave one workgroup a CU (8192 rows, rank 128, 4096 x 4096: 250 against 261 us),
    // which pays with 64 places only (below).
    y.rt = y.mt == 1 && y.slots * blocks <= 1024 ? 1 : blocks >= 4 && !grad ? 4 : blocks >= 2 ? 2 : 1;
    // 64 places by 64 ranks where that makes a workgroup for each CU (8192 rows, rank 64, K = 4096,
    // 133 of them: 30 us, with 32 places 25).
    y.st = y.mt == 1 ? 1 : 2;
    if (y.mt == 4 && blocks >= 3 && y.slots * ((blocks + 3) / 4) * (grad ? 2 : 1) >= 256) y.st = y.rt = 4;
    // Where CUs idle, several workgroups share a tile's K, 2 steps a wave at least (8 rows of
    // their own adapters, rank 16, K = 14336: 10.3 us, unshared 14.9; 64 rows, K = 4096: 10.9 and
    // 11.9).
    y.splits = 1;
    if (!grad && y.mt == 1 && y.rt == 1)
        while (y.splits < MAX_SPLITS && y.slots * blocks * y.splits * 2 <= 256 && K >= (int64_t)SHRINK_STEP * 16 * 2 * y.splits * 2) y.splits *= 2;
    y.chunk = 0;
    y.units = groups;
    // Sums over places: a group at a time, or, where that leaves CUs idle and there are places
    // enough to pay for joining, chunks of a group.  A CU holds two workgroups, one of 64 ranks.
    const int64_t tiles = ((N + 127) / 128 + (K + 127) / 128) * ((blocks + 3) / 4), want = blocks >= 3 ? 256 : 512;
    if (grad && tiles * groups < want && rows > 2048) {
        const int64_t splits = (want + tiles - 1) / tiles;
        y.chunk = (int)std::max<int64_t>(512, round_up((rows + splits - 1) / splits, 128));
        y.units = row_tiles(y.chunk, rows, groups, true);
    }
    // Small groups that are many have work for 2 waves each; where CUs idle, 8 finish sooner (515
    // rows by 5 groups, 1000 x 520: 8 us, with 2 waves 14).
    y.outer_waves = rows <= 128 * (int64_t)groups && tiles * groups >= 1024 ? 2 : 8;
    return y;
}

size_t place_words(const Layout &y) { return (size_t)y.slots * y.mt * 16 * y.ranks; }

template <int T, int MT, int RT>
void launch_shrink(const ShrinkArgs &a, const Layout &y, int deep, hipStream_t s) {
    const dim3 grid((unsigned)(round_up(y.slots, 8) * (y.mt / MT)), (unsigned)((y.ranks / 16 + RT - 1) / RT), deep);
    const dim3 block(64 * shrink_waves(MT, RT));
    if constexpr (RT < 4 || MT == 4)  // the gradients' layout has no others
        if (a.job[0].strided) {
            hipLaunchKernelGGL((shrink_kernel<T, MT, RT, true>), grid, block, shrink_lds(MT, RT), s, a);
            return;
        }
    hipLaunchKernelGGL((shrink_kernel<T, MT, RT, false>), grid, block, shrink_lds(MT, RT), s, a);
}
template <int T>
void launch_shrink(ShrinkArgs a, const Layout &y, int deep, hipStream_t s) {
    a.high = 16 * y.mt, a.slots = (int)y.slots, a.splits = y.splits, a.part_words = place_words(y);
    if (y.st == 4) return launch_shrink<T, 4, 4>(a, y, deep, s);
    if (y.st == 1) {
        if (y.rt == 1) return launch_shrink<T, 1, 1>(a, y, deep, s);
        if (y.rt == 2) return launch_shrink<T, 1, 2>(a, y, deep, s);
        return launch_shrink<T, 1, 4>(a, y, deep, s);
    }
    if (y.rt == 1) return launch_shrink<T, 2, 1>(a, y, deep, s);
    if (y.rt == 2) return launch_shrink<T, 2, 2>(a, y, deep, s);
    launch_shrink<T, 2, 4>(a, y, deep, s);
}

template <int T, int OT, int MT, bool STRIDED>
void launch_expand(const ExpandArgs &a, const Layout &y, hipStream_t s) {
    const dim3 grid((unsigned)(y.slots * ((a.N + 255) / 256)));
    const size_t lds = expand_p_words(MT, y.ranks) * 4 + 4 * expand_own_bytes(a.rank);
    if (y.rs == 1)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 1, STRIDED>), grid, dim3(256), lds, s, a);
    else if (y.rs == 2)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 2, STRIDED>), grid, dim3(256), lds, s, a);
    else if (y.rs == 4)
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 4, STRIDED>), grid, dim3(256), lds, s, a);
    else
        hipLaunchKernelGGL((expand_kernel<T, OT, MT, 8, STRIDED>), grid, dim3(256), lds, s, a);
}
template <int T, bool STRIDED>
void launch_expand(const ExpandArgs &a, int32_t otype, const Layout &y, hipStream_t s) {
    if (otype == BAKRON_T_F32)
        y.mt == 1 ? launch_expand<T, BAKRON_T_F32, 1, STRIDED>(a, y, s) : launch_expand<T, BAKRON_T_F32, 4, STRIDED>(a, y, s);
    else
        y.mt == 1 ? launch_expand<T, T, 1, STRIDED>(a, y, s) : launch_expand<T, T, 4, STRIDED>(a, y, s);
}

template <int T, int WAVES, int PARTS>
void launch_outer(const OuterArgs &a, const Layout &y, hipStream_t s) {
    const int64_t across = (std::max(a.job[0].cols, a.job[1].cols) + 127) / 128;
    const int blocks = y.ranks / 16;
    const unsigned x = (unsigned)(across * a.units);
    if (blocks == 1)
        hipLaunchKernelGGL((outer_kernel<T, WAVES, 1, PARTS>), dim3(x, 1, 2), dim3(64 * WAVES), 0, s, a);
    else if (blocks == 2)
        hipLaunchKernelGGL((outer_kernel<T, WAVES, 2, PARTS>), dim3(x, 1, 2), dim3(64 * WAVES), 0, s, a);
    else
        hipLaunchKernelGGL((outer_kernel<T, WAVES, 4, PARTS>), dim3(x, (unsigned)((blocks + 3) / 4), 2), dim3(64 * WAVES), 0, s, a);
}
template <int T>
void launch_outer(const OuterArgs &a, const Layout &y, hipStream_t s) {
    if (parts_of(a.otype) == 3)
        y.outer_waves == 2 ? launch_outer<T, 2, 3>(a, y, s) : launch_outer<T, 8, 3>(a, y, s);
    else
        y.outer_waves == 2 ? launch_outer<T, 2, 2>(a, y, s) : launch_outer<T, 8, 2>(a, y, s);
    if (a.chunk) {
        const int64_t threads = (a.rank * (int64_t)std::max(a.job[0].cols, a.job[1].cols) + 7) / 8;
        hipLaunchKernelGGL(outer_join_kernel, dim3((unsigned)((threads + 255) / 256), a.of.groups, 2), dim3(256), 0, s, a);
    }
}

bool aligned(const void *p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool sizes_ok(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups, bool grad) {
    if (!(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM && rank >= 1 &&
          rank <= MAX_RANK && groups >= 1 && groups <= MAX_GROUPS))
        return false;
    // no launch of 2^32 threads or more in a dimension; expand and outer are the widest
    const int64_t most = std::max(N, K);
    const Layout y = layout_of(rows, N, K, rank, groups, grad);
    return y.slots * ((most + 255) / 256) * 256 <= LAUNCH_THREADS &&
           (!grad || y.units * ((most + 127) / 128) * 64 * y.outer_waves <= LAUNCH_THREADS);
}

int32_t check_common(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups, const int32_t *offsets,
                     int32_t type, bool grad) {
    BK_REQUIRE(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM,
               "bad sizes rows=%lld N=%lld K=%lld", (long long)rows, (long long)N, (long long)K);
    BK_REQUIRE(rank >= 1 && rank <= MAX_RANK, "rank must be in 1 .. %d, not %d", MAX_RANK, rank);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    BK_REQUIRE(sizes_ok(rows, N, K, rank, groups, grad), "too many tiles: rows=%lld N=%lld K=%lld groups=%d", (long long)rows,
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

size_t tiles_size(const Layout &y) { return align256(y.slots * sizeof(Tile)) + align256(y.slots * 16 * y.mt * sizeof(int32_t)); }

size_t grad_size(const Layout &y, int64_t N, int64_t K, int32_t rank, bool x, bool w) {
    size_t n = tiles_size(y);
    if (x) n += align256(place_words(y) * 4);      // U by place
    if (w) n += 2 * align256(place_words(y) * 4);  // U and P by rank
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
    if (!sizes_ok(rows, N, K, rank, groups, false)) return 0;
    const Layout y = layout_of(rows, N, K, rank, groups, false);
    return tiles_size(y) + align256(y.splits * place_words(y) * 4);
}

extern "C" int32_t bakron_adapter_matmul(const void *X, int32_t type, int64_t ldx, const void *A, const void *B,
                                         int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups,
                                         const int32_t *offsets, const int32_t *order, const float *scale,
                                         const void *base, int64_t ldb, void *out, int32_t otype, int64_t ldo,
                                         int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(X && A && B && out, "X, A, B and out must be non-NULL");
    BK_TRY(check_common(rows, N, K, rank, groups, offsets, type, false));
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
    int32_t *place_rows = c.take<int32_t>(y.slots * 16 * y.mt);
    uint32_t *p = c.take<uint32_t>(y.splits * place_words(y));
    ShrinkArgs h = {};
    h.of = of, h.scale = scale, h.rank = rank, h.ranks = y.ranks, h.tiles = tiles, h.rows = place_rows;
    h.job[0] = {static_cast<const char *>(X), static_cast<const char *>(A), ldx, rank * K, (int)K, 0, p, nullptr, parts_of(otype), 0};
    ExpandArgs e = {};
    e.of = of, e.tiles = tiles, e.rows = place_rows, e.splits = y.splits, e.part_words = place_words(y), e.p = p, e.w = static_cast<const char *>(B), e.group_w = N * rank;
    e.base = static_cast<const char *>(base), e.out = static_cast<char *>(out), e.ldb = ldb, e.ldo = ldo;
    e.N = (int)N, e.rank = rank, e.ranks = y.ranks, e.per_chunk = rank < 8 ? 0 : 65535 / (rank / 8) + 1;
    if (type == BAKRON_T_BF16) {
        launch_shrink<BAKRON_T_BF16>(h, y, y.splits, s);
        launch_expand<BAKRON_T_BF16, false>(e, otype, y, s);
    } else {
        launch_shrink<BAKRON_T_F16>(h, y, y.splits, s);
        launch_expand<BAKRON_T_F16, false>(e, otype, y, s);
    }
    BK_LAUNCH_CHECK("adapter product");
    return BAKRON_OK;
}

extern "C" size_t bakron_adapter_matmul_grad_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t rank,
                                                            int32_t groups) {
    if (!sizes_ok(rows, N, K, rank, groups, true)) return 0;
    return grad_size(layout_of(rows, N, K, rank, groups, true), N, K, rank, true, true);
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
    BK_TRY(check_common(rows, N, K, rank, groups, offsets, type, true));
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
    BK_TRY(check_ws(ws, ws_bytes, grad_size(y, N, K, rank, dX, dA)));
    BK_TRY(check_device());
    hipStream_t s = static_cast<hipStream_t>(stream_);
    const Groups of = {offsets, order, groups, rows, dev_status};
    const char *x = static_cast<const char *>(X), *dy = static_cast<const char *>(dY);
    const char *a = static_cast<const char *>(A), *b = static_cast<const char *>(B);
    Carver c(ws);
    Tile *tiles = c.take<Tile>(y.slots);
    int32_t *place_rows = c.take<int32_t>(y.slots * 16 * y.mt);
    uint32_t *u = dX ? c.take<uint32_t>(place_words(y)) : nullptr, *ur = nullptr, *pr = nullptr;
    if (dA) ur = c.take<uint32_t>(place_words(y)), pr = c.take<uint32_t>(place_words(y));
    float *part = dA && y.chunk ? c.take<float>((size_t)y.units * rank * (N + K)) : nullptr;

    ShrinkArgs h = {};
    h.of = of, h.scale = scale, h.rank = rank, h.ranks = y.ranks, h.tiles = tiles, h.rows = place_rows;
    h.job[0] = {dy, b, lddy, N * rank, (int)N, 1, u, ur, parts_of(xtype), parts_of(wtype)};
    h.job[1] = {x, a, ldx, rank * K, (int)K, 0, nullptr, pr, 0, parts_of(wtype)};
    const int jobs = dA ? 2 : 1;
    type == BAKRON_T_BF16 ? launch_shrink<BAKRON_T_BF16>(h, y, jobs, s) : launch_shrink<BAKRON_T_F16>(h, y, jobs, s);

    // X and dY are read again first, while caches may hold them
    if (dA) {
        OuterArgs o = {};
        o.of = of, o.rank = rank, o.ranks = y.ranks, o.high = 16 * y.mt, o.chunk = y.chunk, o.units = (int)y.units;
        o.subs = y.slots * y.mt;
        o.otype = wtype, o.part = part, o.part_size = (int64_t)rank * (N + K);
        o.job[0] = {x, ldx, (int)K, ur, static_cast<char *>(dA), rank * K, 0, 0};
        o.job[1] = {dy, lddy, (int)N, pr, static_cast<char *>(dB), N * rank, 1, rank * K};
        type == BAKRON_T_BF16 ? launch_outer<BAKRON_T_BF16>(o, y, s) : launch_outer<BAKRON_T_F16>(o, y, s);
    }
    if (dX) {
        ExpandArgs e = {};
        e.of = of, e.tiles = tiles, e.rows = place_rows, e.splits = 1, e.p = u, e.w = a, e.group_w = K * rank;
        e.base = static_cast<const char *>(base), e.out = static_cast<char *>(dX), e.ldb = ldb, e.ldo = lddx;
        e.N = (int)K, e.rank = rank, e.ranks = y.ranks;
        type == BAKRON_T_BF16 ? launch_expand<BAKRON_T_BF16, true>(e, xtype, y, s)
                              : launch_expand<BAKRON_T_F16, true>(e, xtype, y, s);
    }
    BK_LAUNCH_CHECK("adapter gradients");
    return BAKRON_OK;
}
