// fp8.hip -- bakron_fp8_quantize and bakron_fp8_from_codes: data in 8-bit
// floating point (e4m3: 4 exponent bits, 3 mantissa bits, largest value 448).
#include "common.hpp"
#include "elem.hpp"
#include "fp8.hpp"

namespace bakron {
namespace {

// A scale for each row and 128 columns.  A wave takes 4 rows x KPW blocks: 16
// lanes hold the 128 columns of one block, 8 each, so a row's part of a block is
// one contiguous stretch and the maximum stays inside a DPP row.  All KPW blocks
// are loaded before the first is used.
constexpr int KPW = 4;

template <int T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(
    const char *__restrict__ X, int64_t rows, int64_t cols, int64_t ldx, uint8_t *__restrict__ Q,
    int64_t ldq, float *__restrict__ scales, int32_t *dev_status) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * 16 + w * 4 + (lane >> 4);
    const int64_t kb0 = (int64_t)blockIdx.y * KPW, nkb = (cols + 127) / 128;
    if (row >= rows) return;  // whole DPP rows leave together
    float x[KPW][8];
#pragma unroll
    for (int p = 0; p < KPW; ++p) {
        const int64_t c = (kb0 + p) * 128 + (lane & 15) * 8;
        load8<T>(X, row * ldx + c, cols - c, x[p]);
    }
    bool any_bad = false;
#pragma unroll
    for (int p = 0; p < KPW; ++p) {
        const int64_t c = (kb0 + p) * 128 + (lane & 15) * 8;
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(x[p][q]) & 0x7fffffffu);
        m = row_max(m);
        float scale, inv;
        bool bad;
        block_scale(m, scale, inv, bad);
        any_bad |= bad;
        if (c < cols) store8(Q + row * ldq + c, encode8(x[p], inv, bad), (int)min<int64_t>(8, cols - c));
        if ((lane & 15) == 0 && kb0 + p < nkb) scales[(kb0 + p) * rows + row] = scale;
    }
    if (any_bad && dev_status && (lane & 15) == 0) atomicOr(dev_status, BAKRON_DEV_NONFINITE);
}

// A scale for each 128 x 128 block: one workgroup a block, 16 lanes across and
// 16 rows at a time, the block held in registers between maximum and store.
template <int T>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(
    const char *__restrict__ X, int64_t rows, int64_t cols, int64_t ldx, uint8_t *__restrict__ Q,
    int64_t ldq, float *__restrict__ scales, int32_t *dev_status) {
    __shared__ uint32_t part[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 128 + (lane & 15) * 8;
    const int64_t r0 = (int64_t)blockIdx.y * 128 + w * 4 + (lane >> 4);
    float x[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + 16 * p;
        load8<T>(X, r * ldx + c, r < rows ? cols - c : 0, x[p]);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(x[p][q]) & 0x7fffffffu);
    m = row_max(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (lane == 0) part[w] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
    float scale, inv;
    bool bad;
    block_scale(m, scale, inv, bad);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + 16 * p;
        if (r < rows && c < cols)
            store8(Q + r * ldq + c, encode8(x[p], inv, bad), (int)min<int64_t>(8, cols - c));
    }
    if (threadIdx.x == 0) {
        scales[(int64_t)blockIdx.x * ((rows + 127) / 128) + blockIdx.y] = scale;
        if (bad && dev_status) atomicOr(dev_status, BAKRON_DEV_NONFINITE);
    }
}

// code - zero as e4m3.  Every code of at most 4 bits gives an integer in
// [-15, 15], which e4m3 holds exactly.  16 codes a thread.
__global__ __launch_bounds__(256) void from_codes_kernel(const int8_t *__restrict__ codes,
                                                         const float *__restrict__ zeros, int64_t m,
                                                         int64_t n, uint8_t *__restrict__ Q,
                                                         int64_t ldq) {
    const int64_t per_row = (n + 15) / 16;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= m * per_row) return;
    const int64_t r = t / per_row, c = (t - r * per_row) * 16;
    const float z = zeros ? zeros[r] : 0.0f;
    const int count = (int)min<int64_t>(16, n - c);
    int8_t in[16] = {};
    const int8_t *src = codes + r * n + c;
    if (count == 16)
        __builtin_memcpy(in, src, 16);
    else
        for (int q = 0; q < count; ++q) in[q] = src[q];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = (float)in[8 * h + q] - z;
        store8(Q + r * ldq + c + 8 * h, encode8(x, 1.0f, false), count - 8 * h);
    }
}

template <int T>
void launch_quantize(const void *X, int64_t rows, int64_t cols, int64_t ldx, int32_t block_rows,
                     uint8_t *Q, int64_t ldq, float *scales, int32_t *dev_status, hipStream_t s) {
    const char *x = static_cast<const char *>(X);
    const int64_t kb = (cols + 127) / 128;
    if (block_rows == 1)
        hipLaunchKernelGGL(quantize_rows_kernel<T>,
                           dim3((unsigned)((rows + 15) / 16), (unsigned)((kb + KPW - 1) / KPW)),
                           dim3(256), 0, s, x, rows, cols, ldx, Q, ldq, scales, dev_status);
    else
        hipLaunchKernelGGL(quantize_blocks_kernel<T>, dim3((unsigned)kb, (unsigned)((rows + 127) / 128)),
                           dim3(256), 0, s, x, rows, cols, ldx, Q, ldq, scales, dev_status);
}

constexpr int64_t MAX_ROWS = int64_t(1) << 22;  // grid limits: rows / 128 and cols / 512 below 65536
constexpr int64_t MAX_COLS = int64_t(1) << 22;

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" int32_t bakron_fp8_quantize(const void *X, int32_t type, int64_t rows, int64_t cols,
                                       int64_t ldx, int32_t block_rows, uint8_t *Q, int64_t ldq,
                                       float *scales, int32_t *dev_status, void *stream_) {
    clear_error();
    BK_REQUIRE(X && Q && scales, "X, Q and scales must be non-NULL");
    BK_REQUIRE(type == BAKRON_T_F32 || type == BAKRON_T_BF16 || type == BAKRON_T_F16, "bad type %d", type);
    BK_REQUIRE(rows >= 1 && cols >= 1 && rows <= MAX_ROWS && cols <= MAX_COLS,
               "bad sizes rows=%lld cols=%lld", (long long)rows, (long long)cols);
    BK_REQUIRE(ldx >= cols && ldq >= cols && ldx <= MAX_LD && ldq <= MAX_LD,
               "bad row strides ldx=%lld ldq=%lld for %lld columns", (long long)ldx, (long long)ldq,
               (long long)cols);
    BK_REQUIRE(block_rows == 1 || block_rows == 128, "block_rows must be 1 or 128, not %d", block_rows);
    BK_REQUIRE((reinterpret_cast<uintptr_t>(X) & (elem_size(type) - 1)) == 0, "X is misaligned for its type");
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    if (type == BAKRON_T_F32)
        launch_quantize<BAKRON_T_F32>(X, rows, cols, ldx, block_rows, Q, ldq, scales, dev_status, s);
    else if (type == BAKRON_T_BF16)
        launch_quantize<BAKRON_T_BF16>(X, rows, cols, ldx, block_rows, Q, ldq, scales, dev_status, s);
    else
        launch_quantize<BAKRON_T_F16>(X, rows, cols, ldx, block_rows, Q, ldq, scales, dev_status, s);
    BK_LAUNCH_CHECK("fp8 quantisation");
    return BAKRON_OK;
}

extern "C" int32_t bakron_fp8_from_codes(const int8_t *codes, const float *zeros, int64_t m, int64_t n,
                                         int32_t qkind, int32_t qbits, uint8_t *Q, int64_t ldq,
                                         void *stream_) {
    clear_error();
    BK_REQUIRE(codes && Q, "codes and Q must be non-NULL");
    BK_REQUIRE(m >= 1 && n >= 1 && m <= MAX_ROWS && n <= MAX_COLS && m * n <= (int64_t(1) << 40),
               "bad sizes m=%lld n=%lld", (long long)m, (long long)n);
    BK_REQUIRE(ldq >= n && ldq <= MAX_LD, "bad row stride ldq=%lld for %lld columns", (long long)ldq,
               (long long)n);
    BK_REQUIRE((qkind == BAKRON_Q_SYM || qkind == BAKRON_Q_ASYM) && qbits >= 2 && qbits <= 4,
               "codes of kind %d with %d bits are not all exact in e4m3", qkind, qbits);
    BK_REQUIRE((qkind == BAKRON_Q_ASYM) == (zeros != nullptr),
               "zeros go with asymmetric codes, and only with them");
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    const int64_t per_row = (n + 15) / 16, most = (LAUNCH_THREADS - 255) / per_row;  // rows of a launch
    for (int64_t r = 0; r < m; r += most) {
        const int64_t rows = m - r < most ? m - r : most;
        hipLaunchKernelGGL(from_codes_kernel, dim3((unsigned)((rows * per_row + 255) / 256)), dim3(256), 0,
                           static_cast<hipStream_t>(stream_), codes + r * n, zeros ? zeros + r : nullptr, rows, n,
                           Q + r * ldq, ldq);
        BK_LAUNCH_CHECK("from_codes_kernel");
    }
    return BAKRON_OK;
}
