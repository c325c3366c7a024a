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
#include "common.hpp"
#include "elem.hpp"

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
    int vec;                 // 1: rows of C start on 4-element boundaries
};

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
    int x = (int)v;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    return x;
}

// Group g's rows [a, b), kept inside [0, rows) whatever the offsets hold.  Group
// `groups` stands for the rows after the last group.
__device__ __forceinline__ void group_range(const ProductArgs &p, int g, int64_t &a, int64_t &b) {
    if (!p.offsets) {
        a = g == 0 ? 0 : p.rows;
        b = p.rows;
        return;
    }
    a = g == 0 ? 0 : min<int64_t>(max<int64_t>(p.offsets[g], 0), p.rows);
    b = g == p.groups ? p.rows : min<int64_t>(max<int64_t>(p.offsets[g + 1], a), p.rows);
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

// Workgroups are dealt to the 8 XCDs in turn: XCD x takes the x-th eighth of the
// work, so that tiles that share operands share an L2.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t total) {
    const int64_t q = total >> 3, r = total & 7, x = b & 7;
    return x * q + min(x, r) + (b >> 3);
}

// Finds the workgroup's rows: tiles of BI rows are counted group by group, then
// walked in bands of 8 row tiles.  All 64 lanes of a wave take part.  False: no
// work for this workgroup.
template <int BI>
__device__ __forceinline__ bool find_rows(const ProductArgs &p, int64_t b, int &g, int64_t &i0, int64_t &i1,
                                          int &tj) {
    const int lane = threadIdx.x & 63;
    int64_t slots = 0;
    if (!p.offsets) {
        slots = (p.rows + BI - 1) / BI;
    } else {
        int64_t mine = 0;
        for (int e = lane; e <= p.groups; e += 64) {
            int64_t a, z;
            group_range(p, e, a, z);
            mine += (z - a + BI - 1) / BI;
        }
        slots = wave_sum(mine);
    }
    const int64_t total = slots * p.tiles_j;
    if (b >= total) return false;
    const int64_t w = xcd_order(b, total);
    const int64_t per_band = 8 * (int64_t)p.tiles_j;
    const int64_t band = w / per_band, in = w - band * per_band;
    const int64_t width = min<int64_t>(8, slots - band * 8);
    int64_t slot = band * 8 + in % width;
    tj = (int)(in / width);
    if (!p.offsets) {
        g = 0;
        i0 = slot * BI;
        i1 = min<int64_t>(p.rows, i0 + BI);
        return true;
    }
    for (int base = 0; base <= p.groups; base += 64) {
        const int e = base + lane;
        int64_t a = 0, z = 0;
        if (e <= p.groups) group_range(p, e, a, z);
        const int mine = (int)((z - a + BI - 1) / BI);
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(upto, off);
            if (lane >= off) upto += v;
        }
        const uint64_t hit = __ballot(slot < upto);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            g = base + src;
            group_range(p, g, a, z);
            const int before = __shfl(upto - mine, src);
            i0 = a + (slot - before) * BI;
            i1 = min<int64_t>(z, i0 + BI);
            g = __builtin_amdgcn_readfirstlane(g);
            return true;
        }
        slot -= __shfl(upto, 63);
    }
    return false;
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
    static __device__ __forceinline__ int swap(int r) { return (r & 3) | ((r >> 1) & 4); }

    // where the chunk at LDS place q comes from: row (of the tile, or of r) and byte in it
    static __device__ __forceinline__ void place(int q, int &row, int &byte) {
        row = q / (ROW / 16);
        const int c = q % (ROW / 16);
        if constexpr (STRIDED)
            byte = (((c >> 1) ^ swap(row)) << 5) | ((c & 1) << 4);
        else
            byte = (c ^ (row & 7)) << 4;
    }

    // byte address of the lane's first 8 bytes (strided) or 16 bytes for tile columns
    // c0 .. c0 + 15 and half h (32 of 64 values of r; for fp8 64 of 128)
    static __device__ __forceinline__ int frag(int c0, int h, int lane) {
        const int l = lane & 15, g = lane >> 4;
        if constexpr (STRIDED) {
            const int r = 32 * h + 8 * g + (l >> 2);
            return r * ROW + (((c0 >> 4) ^ swap(r)) << 5) + (l & 3) * 8;
        } else {
            const int n = c0 + l;
            return n * STEP + (((4 * h + g) ^ (n & 7)) << 4);
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
__device__ __forceinline__ floatx4 mfma_f8(intx4 a0, intx4 a1, intx4 b0, intx4 b1) {
    const intx8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const intx8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    const floatx4 zero = {0, 0, 0, 0};
    // format 0 = e4m3 on both sides; all block exponents 2^0
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ void put4(const ProductArgs &p, int64_t at, int64_t left, floatx4 v) {
    if (p.ytype == BAKRON_T_F32) {
        float *y = reinterpret_cast<float *>(p.Y) + at;
        if (left >= 4 && p.vec)
            *reinterpret_cast<floatx4 *>(y) = v;
        else
            for (int q = 0; q < 4 && q < left; ++q) y[q] = v[q];
        return;
    }
    uint32_t w[2];
    if (p.ytype == BAKRON_T_BF16)
        w[0] = pack2<BAKRON_T_BF16>(v[0], v[1]), w[1] = pack2<BAKRON_T_BF16>(v[2], v[3]);
    else
        w[0] = pack2<BAKRON_T_F16>(v[0], v[1]), w[1] = pack2<BAKRON_T_F16>(v[2], v[3]);
    uint16_t *y = reinterpret_cast<uint16_t *>(p.Y) + at;
    if (left >= 4 && p.vec)
        *reinterpret_cast<uint2 *>(y) = make_uint2(w[0], w[1]);
    else
        for (int q = 0; q < 4 && q < left; ++q) y[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
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

    report_offsets(p);
    int g, tj;
    int64_t i0, i1, R = p.R;
    const char *P = p.P, *Q = p.Q;
    int64_t yoff = 0;
    if constexpr (MODE == GRAD_W) {
        const int64_t tiles = (int64_t)p.tiles_i * p.tiles_j, w = xcd_order(blockIdx.x, tiles * p.groups);
        g = (int)(w / tiles);
        const int t = (int)(w - g * tiles);
        tj = t / p.tiles_i;
        i0 = (int64_t)(t % p.tiles_i) * BI;
        i1 = min<int64_t>(p.I, i0 + BI);
        int64_t a, b;
        group_range(p, g, a, b);
        R = b - a;
        P += a * p.ldp;
        Q += a * p.ldq;
        yoff = g * p.group_y;
    } else {
        if (!find_rows<BI>(p, blockIdx.x, g, i0, i1, tj)) return;
        if (g == p.groups)
            R = 0;  // rows of no group
        else
            Q += g * p.group_q;
    }
    const int64_t j0 = (int64_t)tj * BJ;
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
                sc[a] = p.sp[s * p.rows + min<int64_t>(i, i1 - 1)];
            }
            if constexpr (SCALE == BAKRON_SCALE_BLOCK) {
                // a wave's columns lie in one block of 128
                const int64_t nb = (p.J + 127) / 128;
                const int64_t jb = min<int64_t>((j0 + wj * (BJ / WJ)) / 128, nb - 1);
                const float w = p.sq[((int64_t)g * steps + s) * nb + jb];
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
                    const floatx4 t = mfma_f8(q0, q1, fp[a][0], fp[a][1]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[a][b][v] = fmaf(sc[a], t[v], acc[a][b][v]);
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

#pragma unroll
    for (int b = 0; b < NJ; ++b) {
        const int64_t j = j0 + wj * (BJ / WJ) + b * 16 + 4 * (lane >> 4);
        floatx4 w = {1, 1, 1, 1};
        if constexpr (SCALE == BAKRON_SCALE_ROW) {
            if (g < p.groups)
                for (int v = 0; v < 4; ++v)
                    if (j + v < p.J) w[v] = p.sq[g * p.J + j + v];
        }
#pragma unroll
        for (int a = 0; a < NI; ++a) {
            const int64_t i = i0 + wi * (BI / WI) + a * 16 + (lane & 15);
            floatx4 t = acc[a][b];
            if constexpr (SCALE == BAKRON_SCALE_ROW)
                for (int v = 0; v < 4; ++v) t[v] *= w[v];
            if (i < i1 && j < p.J) put4(p, yoff + i * p.ldy + j, p.J - j, t);
        }
    }
}

constexpr int64_t MAX_DIM = int64_t(1) << 24;
constexpr int32_t MAX_GROUPS = 4096;

template <int ET, int MODE, int SCALE>
void launch(ProductArgs &p, hipStream_t s) {
    constexpr int BI = 128, BJ = 128;
    p.tiles_j = (int)((p.J + BJ - 1) / BJ);
    p.tiles_i = (int)((p.I + BI - 1) / BI);
    int64_t grid;
    if constexpr (MODE == GRAD_W)
        grid = (int64_t)p.groups * p.tiles_i * p.tiles_j;
    else
        grid = ((p.rows + BI - 1) / BI + (p.offsets ? p.groups + 1 : 0)) * p.tiles_j;
    hipLaunchKernelGGL((product_kernel<ET, MODE, SCALE, BI, BJ, 2, 2>), dim3((unsigned)grid), dim3(256), 0, s, p);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Limits that keep every index in range: no size over 2^24, no more than 2^31
// workgroups of the smallest tiles.
int32_t check_sizes(int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets) {
    BK_REQUIRE(rows >= 1 && N >= 1 && K >= 1 && rows <= MAX_DIM && N <= MAX_DIM && K <= MAX_DIM,
               "bad sizes rows=%lld N=%lld K=%lld", (long long)rows, (long long)N, (long long)K);
    BK_REQUIRE(groups >= 1 && groups <= MAX_GROUPS, "groups must be in 1 .. %d, not %d", MAX_GROUPS, groups);
    BK_REQUIRE(offsets || groups == 1, "offsets must be non-NULL for %d groups", groups);
    BK_REQUIRE((rows / 16 + 1 + groups + 1) * (N / 16 + 1) < (int64_t(1) << 31) &&
                   (rows / 16 + 1 + groups + 1) * (K / 16 + 1) < (int64_t(1) << 31) &&
                   (int64_t)groups * (N / 64 + 1) * (K / 64 + 1) < (int64_t(1) << 31),
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
    return ld % 4 == 0 && aligned(Y, 4 * elem_size(ytype));
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
    (void)rows, (void)N, (void)K, (void)groups;
    return 0;
}

extern "C" size_t bakron_grouped_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t groups) {
    (void)rows, (void)N, (void)K, (void)groups;
    return 0;
}

extern "C" int32_t bakron_fp8_matmul(const uint8_t *X, int64_t ldx, const float *sx, const uint8_t *W,
                                     int64_t ldw, const float *sw, int32_t wscale, int64_t rows, int64_t N,
                                     int64_t K, int32_t groups, const int32_t *offsets, void *Y,
                                     int32_t ytype, int64_t ldy, int32_t *dev_status, void *ws,
                                     size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(X && sx && W && sw && Y, "X, sx, W, sw and Y must be non-NULL");
    BK_REQUIRE(wscale == BAKRON_SCALE_ROW || wscale == BAKRON_SCALE_BLOCK, "bad weight scale kind %d", wscale);
    BK_TRY(check_sizes(rows, N, K, groups, offsets));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("ldy", ldy, N, rows));
    BK_TRY(check_type16(ytype));
    BK_TRY(check_out(Y, ytype, ytype));
    (void)ws;
    (void)ws_bytes;
    BK_TRY(check_device());
    ProductArgs p = {};
    p.P = reinterpret_cast<const char *>(X), p.Q = reinterpret_cast<const char *>(W);
    p.Y = static_cast<char *>(Y);
    p.ldp = ldx, p.ldq = ldw, p.ldy = ldy, p.group_q = ldw * N;
    p.sp = sx, p.sq = sw;
    p.rows = p.I = rows, p.J = N, p.R = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = ytype;
    p.vec = vector_rows(Y, ytype, ldy);
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
    BK_TRY(check_sizes(rows, N, K, groups, offsets));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("ldy", ldy, N, rows));
    BK_TRY(check_out(Y, ytype, type));
    BK_REQUIRE(aligned(X, 2) && aligned(W, 2), "X or W is misaligned for its type");
    (void)ws;
    (void)ws_bytes;
    BK_TRY(check_device());
    ProductArgs p = {};
    p.P = static_cast<const char *>(X), p.Q = static_cast<const char *>(W), p.Y = static_cast<char *>(Y);
    p.ldp = 2 * ldx, p.ldq = 2 * ldw, p.ldy = ldy, p.group_q = 2 * ldw * N;
    p.rows = p.I = rows, p.J = N, p.R = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = ytype;
    p.vec = vector_rows(Y, ytype, ldy);
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
    BK_TRY(check_sizes(rows, N, K, groups, offsets));
    BK_TRY(check_ld("lddy", lddy, N, rows));
    BK_TRY(check_ld("ldw", ldw, K, groups * N));
    BK_TRY(check_ld("lddx", lddx, K, rows));
    BK_TRY(check_out(dX, dxtype, type));
    BK_REQUIRE(aligned(dY, 2) && aligned(W, 2), "dY or W is misaligned for its type");
    (void)ws;
    (void)ws_bytes;
    BK_TRY(check_device());
    ProductArgs p = {};
    p.P = static_cast<const char *>(dY), p.Q = static_cast<const char *>(W), p.Y = static_cast<char *>(dX);
    p.ldp = 2 * lddy, p.ldq = 2 * ldw, p.ldy = lddx, p.group_q = 2 * ldw * N;
    p.rows = p.I = rows, p.J = K, p.R = N;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = dxtype;
    p.vec = vector_rows(dX, dxtype, lddx);
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
    BK_TRY(check_sizes(rows, N, K, groups, offsets));
    BK_TRY(check_ld("lddy", lddy, N, rows));
    BK_TRY(check_ld("ldx", ldx, K, rows));
    BK_TRY(check_ld("lddw", lddw, K, groups * N));
    BK_TRY(check_out(dW, dwtype, type));
    BK_REQUIRE(aligned(dY, 2) && aligned(X, 2), "dY or X is misaligned for its type");
    (void)ws;
    (void)ws_bytes;
    BK_TRY(check_device());
    ProductArgs p = {};
    p.P = static_cast<const char *>(dY), p.Q = static_cast<const char *>(X), p.Y = static_cast<char *>(dW);
    p.ldp = 2 * lddy, p.ldq = 2 * ldx, p.ldy = lddw, p.group_y = lddw * N;
    p.rows = rows, p.I = N, p.J = K;
    p.groups = groups, p.offsets = offsets, p.dev_status = dev_status, p.ytype = dwtype;
    p.vec = vector_rows(dW, dwtype, lddw);
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == BAKRON_T_BF16)
        launch<BAKRON_T_BF16, GRAD_W, SCALE_NONE>(p, s);
    else
        launch<BAKRON_T_F16, GRAD_W, SCALE_NONE>(p, s);
    BK_LAUNCH_CHECK("the grouped product's gradient");
    return BAKRON_OK;
}
