// logprobs.hip -- bakron_token_logprobs and its gradient.
//
// For a row of logits x over a vocabulary of V tokens, with m = max x,
// s = sum e^(x - m) and t = sum e^(x - m) (x - m):
//   lse = m + log s,  log p_j = x_j - lse,  H = -sum p log p = log s - t / s.
// One pass over the row keeps (m, s, t) and rescales the two sums where the
// maximum grows; sums and statistics are fp32.
//
// Alternatives (the k largest, equal values by lowest index).  Each thread reads
// chunks of 16 consecutive elements and leaves each chunk's maximum in LDS.  An
// element of the k largest lies in one of the k chunks that come first by
// (maximum, lowest chunk): any other chunk has k chunks before it, each with an
// element that is larger, or equal at a lower index.  So after the pass only k
// chunks are read again (from L2).  The selections are by counting: the rank of
// a key among a short list is the number of keys above it.
#include "common.hpp"
#include "elem.hpp"

namespace bakron {
namespace {

constexpr int NT = 512;            // threads of a row pass
constexpr int CE = 16;             // elements of a chunk
constexpr int SEG_CHUNKS = 8192;   // chunks of a row that one workgroup takes: 32 KB of maxima
constexpr int64_t SEG = (int64_t)SEG_CHUNKS * CE;
constexpr int KMAX = 64;
constexpr int CAP = 1024;          // candidates held in LDS

struct Stats {
    float m, s, t;
};

// Statistics of the union of two sets.  A set whose weight vanishes adds nothing
// (its m may be so far below that the difference is infinite).
__device__ __forceinline__ Stats merge(Stats a, Stats b) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m - m, db = b.m - m;
    const float ca = __expf(da), cb = __expf(db);
    Stats r;
    r.m = m;
    r.s = ca * a.s + cb * b.s;
    r.t = ca * (a.t + a.s * fmaxf(da, -200.0f)) + cb * (b.t + b.s * fmaxf(db, -200.0f));
    return r;
}

// Order of the values as unsigned integers: NaN above everything, -0 = +0.
__device__ __forceinline__ uint32_t order(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// Larger value first, then lower position.  0 is below every key.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t pos) {
    return ((uint64_t)order(x) << 32) | (uint32_t)~pos;
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int mask) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, mask);
    const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), mask);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ Stats wave_stats(Stats a) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        Stats b;
        b.m = __shfl_xor(a.m, off);
        b.s = __shfl_xor(a.s, off);
        b.t = __shfl_xor(a.t, off);
        a = merge(a, b);
    }
    return a;
}

// The k best of list[0, n) (distinct keys, n <= CAP; 0 entries are none) into
// out[0, k) in order; places without a key get 0.
__device__ __forceinline__ void rank_select(const uint64_t *list, int n, uint64_t *out, int k) {
    for (int i = threadIdx.x; i < k; i += blockDim.x) out[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint64_t key = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += list[j] > key;
        if (rank < k && key) out[rank] = key;
    }
    __syncthreads();
}

struct RowArgs {
    const char *x;
    int64_t rows, vocab, ld;
    const int64_t *targets;
    int k, segs;
    int64_t seg;  // elements of a segment, a multiple of CE
    float *logprob, *lse, *entropy, *top_logprob;
    int64_t *top_ids;
    int32_t *dev_status;
    Stats *part;         // [rows][segs]
    uint64_t *part_top;  // [rows][segs][k]
};

// What a row's statistics give; one thread.
template <int T>
__device__ __forceinline__ float finish_row(const RowArgs &a, int64_t row, Stats st) {
    const bool none = st.s == 0.0f;                    // every logit is -inf
    const bool bad = st.s != st.s || st.m > 3.4028235e38f;  // a NaN or +inf
    const float nan = __uint_as_float(0x7fc00000u);
    const float logs = __logf(st.s);
    float lse = none ? -INFINITY : st.m + logs;
    float ent = none ? 0.0f : logs - st.t / st.s;
    if (bad) lse = ent = nan;
    int32_t flag = bad ? BAKRON_DEV_NONFINITE : 0;
    a.lse[row] = lse;
    a.entropy[row] = ent;
    const int64_t t = a.targets[row];
    float lp = 0.0f;
    if (t >= a.vocab) {
        lp = nan;
        flag |= BAKRON_DEV_BAD_INDEX;
    } else if (t >= 0) {
        lp = none ? -INFINITY : load1<T>(a.x, row * a.ld + t) - lse;
    }
    a.logprob[row] = lp;
    if (flag && a.dev_status) atomicOr(a.dev_status, flag);
    return lse;
}

__device__ __forceinline__ void write_top(const RowArgs &a, int64_t row, const uint64_t *best, float lse) {
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
        const uint64_t key = best[i];
        const float x = unorder((uint32_t)(key >> 32));
        a.top_logprob[row * a.k + i] = lse == -INFINITY ? -INFINITY : x - lse;
        a.top_ids[row * a.k + i] = (int64_t)(uint32_t)~(uint32_t)key;
    }
}

// The k best elements of one segment, from its chunks' maxima cmax[0, nchunk).
template <int T>
__device__ void segment_top(const RowArgs &a, int64_t base, int64_t e0, int64_t e1, const float *cmax,
                            int nchunk, uint64_t *list, uint64_t *best, uint64_t *shared_key, int *count) {
    const int k = a.k, tid = threadIdx.x;
    // a lower bound of the k-th best chunk: the k-th of 64 groups' best chunks
    uint64_t mine = 0;
    for (int c = tid; c < nchunk; c += NT) mine = max64(mine, key_of(cmax[c], (uint32_t)c));
    uint64_t grp = mine;
    grp = max64(grp, shfl_xor64(grp, 1));
    grp = max64(grp, shfl_xor64(grp, 2));
    grp = max64(grp, shfl_xor64(grp, 4));
    if ((tid & 7) == 0) list[tid >> 3] = grp;
    if (tid == 0) *shared_key = 0, *count = 0;
    __syncthreads();
    if (tid < 64) {
        const uint64_t key = list[tid];
        int rank = 0;
        for (int j = 0; j < 64; ++j) rank += list[j] > key;
        if (rank == k - 1 && key) *shared_key = key;  // keys other than 0 are distinct
    }
    __syncthreads();
    const uint64_t bound = *shared_key;
    __syncthreads();
    if (grp >= bound && grp)
        for (int c = tid; c < nchunk; c += NT) {
            const uint64_t key = key_of(cmax[c], (uint32_t)c);
            if (key >= bound) {
                const int at = atomicAdd(count, 1);
                if (at < CAP) list[at] = key;
            }
        }
    __syncthreads();
    const int n = *count;
    if (n <= CAP) {
        rank_select(list, n, best, k);
    } else {
        // far more chunks above the bound than usual: one by one
        uint64_t last = ~0ull;
        for (int i = 0; i < k; ++i) {
            uint64_t top = 0;
            for (int c = tid; c < nchunk; c += NT) {
                const uint64_t key = key_of(cmax[c], (uint32_t)c);
                if (key < last) top = max64(top, key);
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) top = max64(top, shfl_xor64(top, off));
            if ((tid & 63) == 0) list[tid >> 6] = top;
            __syncthreads();
            for (int j = 0; j < NT / 64; ++j) top = max64(top, list[j]);
            if (tid == 0) best[i] = top;
            last = top;
            __syncthreads();
        }
    }
    // the elements of the k chunks that reach the k-th chunk's maximum
    const uint64_t floor = best[k - 1] >> 32;
    if (tid == 0) *count = 0;
    __syncthreads();
    for (int i = tid; i < k * CE; i += NT) {
        const uint64_t ck = best[i / CE];
        const int64_t e = e0 + (int64_t)(uint32_t)~(uint32_t)ck * CE + i % CE;
        if (ck && e < e1) {
            const uint64_t key = key_of(load1<T>(a.x, base + e), (uint32_t)e);
            if ((key >> 32) >= floor) list[atomicAdd(count, 1)] = key;  // k CE <= CAP
        }
    }
    __syncthreads();
    rank_select(list, *count, best, k);
}

// One segment of one row.
template <int T>
__global__ __launch_bounds__(NT) void row_kernel(RowArgs a) {
    __shared__ float cmax[SEG_CHUNKS];
    __shared__ uint64_t list[CAP], best[KMAX], shared_key;
    __shared__ Stats wave_part[NT / 64];
    __shared__ int count;
    __shared__ float row_lse;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.segs, sg = blockIdx.x - row * a.segs;
    const int64_t e0 = sg * a.seg, e1 = min(a.vocab, e0 + a.seg);
    const int nchunk = (int)((e1 - e0 + CE - 1) / CE);
    const int64_t base = row * a.ld;
    Stats st = {-3.4028235e38f, 0.0f, 0.0f};
    for (int c = tid; c < nchunk; c += NT) {
        const int64_t e = e0 + (int64_t)c * CE;
        float x[CE];
        if (e + CE <= e1) {
            load8<T>(a.x, base + e, 8, x);
            load8<T>(a.x, base + e + 8, 8, x + 8);
        } else {
#pragma unroll
            for (int q = 0; q < CE; ++q) x[q] = e + q < e1 ? load1<T>(a.x, base + e + q) : -INFINITY;
        }
        float cm = x[0];
#pragma unroll
        for (int q = 1; q < CE; ++q) cm = fmaxf(cm, x[q]);
        cmax[c] = cm;
        if (cm > st.m) {
            const float d = st.m - cm, f = __expf(d);
            st.t = f * (st.t + st.s * fmaxf(d, -200.0f));
            st.s *= f;
            st.m = cm;
        }
#pragma unroll
        for (int q = 0; q < CE; ++q) {
            const float d = x[q] - st.m;  // NaN stays NaN in the sum s
            const float e1x = __expf(d);
            st.s += e1x;
            st.t += e1x * fmaxf(d, -200.0f);  // 0 where e^d vanishes, for d = -inf too
        }
    }
    st = wave_stats(st);
    if ((tid & 63) == 0) wave_part[tid >> 6] = st;
    __syncthreads();
    if (tid == 0) {
        st = wave_part[0];
        for (int i = 1; i < NT / 64; ++i) st = merge(st, wave_part[i]);
        if (a.segs == 1)
            row_lse = finish_row<T>(a, row, st);
        else
            a.part[blockIdx.x] = st;
    }
    if (a.k == 0) return;
    __syncthreads();
    segment_top<T>(a, base, e0, e1, cmax, nchunk, list, best, &shared_key, &count);
    if (a.segs == 1)
        write_top(a, row, best, row_lse);
    else
        for (int i = tid; i < a.k; i += NT) a.part_top[(int64_t)blockIdx.x * a.k + i] = best[i];
}

// Joins a row's segments, in their order.
template <int T>
__global__ __launch_bounds__(256) void join_kernel(RowArgs a) {
    __shared__ uint64_t list[CAP], best[KMAX], bound;
    __shared__ int count;
    __shared__ float row_lse;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    if (tid == 0) {
        Stats st = a.part[row * a.segs];
        for (int i = 1; i < a.segs; ++i) st = merge(st, a.part[row * a.segs + i]);
        row_lse = finish_row<T>(a, row, st);
        count = 0;
        // the best of the segments' k-th keys is a lower bound of the row's k-th
        uint64_t b = 0;
        for (int i = 0; i < a.segs && a.k; ++i)
            b = max64(b, a.part_top[(row * a.segs + i) * a.k + a.k - 1]);
        bound = b;
    }
    if (a.k == 0) return;
    __syncthreads();
    const int total = a.segs * a.k;
    const uint64_t *top = a.part_top + row * total;
    // total <= CAP, so the list holds every key
    for (int i = tid; i < total; i += 256)
        if (top[i] >= bound && top[i]) list[atomicAdd(&count, 1)] = top[i];
    __syncthreads();
    rank_select(list, count, best, a.k);
    write_top(a, row, best, row_lse);
}

// d logits = -p (g + g_H (log p + H)), and g more at the target.
template <int T>
__global__ __launch_bounds__(256) void grad_kernel(const char *__restrict__ x, int64_t vocab, int64_t ld,
                                                   const int64_t *__restrict__ targets,
                                                   const float *__restrict__ lse,
                                                   const float *__restrict__ entropy,
                                                   const float *__restrict__ g_logprob,
                                                   const float *__restrict__ g_entropy,
                                                   char *__restrict__ dx, int64_t ldd, int segs,
                                                   int32_t *dev_status) {
    const int64_t row = blockIdx.x / segs, sg = blockIdx.x - row * segs;
    const int64_t t = targets[row];
    const float l = lse[row];
    const float g = t >= 0 ? g_logprob[row] : 0.0f, gh = g_entropy ? g_entropy[row] : 0.0f;
    const float h = entropy && g_entropy ? entropy[row] : 0.0f;
    const bool none = l == -INFINITY;  // no distribution: no gradient
    if (t >= vocab && dev_status && sg == 0 && threadIdx.x == 0) atomicOr(dev_status, BAKRON_DEV_BAD_INDEX);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int64_t e = sg * 8192 + p * 2048 + threadIdx.x * 8;
        if (e >= vocab) return;
        float v[8];
        load8<T>(x, row * ld + e, vocab - e, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float lp = v[q] - l;
            const float pr = __expf(lp);
            float d = -pr * (g + gh * (fmaxf(lp, -200.0f) + h));
            if (e + q == t) d += g;
            v[q] = none ? 0.0f : d;
        }
        store8<T>(dx, row * ldd + e, vocab - e, v);
    }
}

// Elements of a segment: a whole row, or less where there are too few rows to
// give every CU work (512 workgroups), but no less than 8192.
int64_t segment_of(int64_t rows, int64_t vocab, int32_t k) {
    const int64_t want = rows >= 512 ? 1 : (512 + rows - 1) / rows;
    int64_t segs = vocab / 8192 < want ? vocab / 8192 : want;
    const int64_t most = k > 0 ? CAP / k : 64;  // the join's list
    if (segs > most) segs = most;
    if (segs < 1) segs = 1;
    int64_t seg = round_up((vocab + segs - 1) / segs, CE);
    return seg < SEG ? seg : SEG;
}

constexpr int64_t MAX_VOCAB = SEG * (CAP / KMAX);  // 2^21
constexpr int64_t MAX_ROWS = int64_t(1) << 24;

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" size_t bakron_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t k) {
    if (rows < 1 || rows > MAX_ROWS || vocab < 1 || vocab > MAX_VOCAB || k < 0 || k > KMAX || k > vocab) return 0;
    const int64_t seg = segment_of(rows, vocab, k), segs = (vocab + seg - 1) / seg;
    if (segs == 1) return 0;
    return align256(rows * segs * sizeof(Stats)) + align256(rows * segs * k * sizeof(uint64_t));
}

extern "C" int32_t bakron_token_logprobs(const void *logits, int32_t type, int64_t rows, int64_t vocab,
                                         int64_t ld, const int64_t *targets, int32_t k, float *logprob,
                                         float *lse, float *entropy, float *top_logprob, int64_t *top_ids,
                                         int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(logits && targets && logprob && lse && entropy,
               "logits, targets, logprob, lse and entropy must be non-NULL");
    BK_REQUIRE(type == BAKRON_T_F32 || type == BAKRON_T_BF16 || type == BAKRON_T_F16, "bad type %d", type);
    BK_REQUIRE(rows >= 1 && rows <= MAX_ROWS && vocab >= 1 && vocab <= MAX_VOCAB,
               "bad sizes rows=%lld vocab=%lld", (long long)rows, (long long)vocab);
    BK_REQUIRE(ld >= vocab && ld <= MAX_LD, "bad row stride ld=%lld for a vocabulary of %lld", (long long)ld,
               (long long)vocab);
    BK_REQUIRE(k >= 0 && k <= KMAX && k <= vocab, "k must be in 0 .. min(%d, vocab), not %d", KMAX, k);
    BK_REQUIRE(k == 0 || (top_logprob && top_ids), "top_logprob and top_ids must be non-NULL for k > 0");
    BK_REQUIRE((reinterpret_cast<uintptr_t>(logits) & (elem_size(type) - 1)) == 0,
               "logits are misaligned for their type");
    RowArgs a = {};
    a.seg = segment_of(rows, vocab, k);
    a.segs = (int)((vocab + a.seg - 1) / a.seg);
    const size_t need = bakron_token_logprobs_workspace_size(rows, vocab, k);
    if (need && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255))) {
        set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, ws_bytes);
        return BAKRON_ERR_WORKSPACE;
    }
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    a.x = static_cast<const char *>(logits);
    a.rows = rows, a.vocab = vocab, a.ld = ld, a.targets = targets, a.k = k;
    a.logprob = logprob, a.lse = lse, a.entropy = entropy;
    a.top_logprob = top_logprob, a.top_ids = top_ids, a.dev_status = dev_status;
    if (a.segs > 1) {
        Carver c(ws);
        a.part = c.take<Stats>(rows * a.segs);
        a.part_top = c.take<uint64_t>(rows * a.segs * k);
    }
    const dim3 grid((unsigned)(rows * a.segs));
    if (type == BAKRON_T_F32)
        hipLaunchKernelGGL(row_kernel<BAKRON_T_F32>, grid, dim3(NT), 0, s, a);
    else if (type == BAKRON_T_BF16)
        hipLaunchKernelGGL(row_kernel<BAKRON_T_BF16>, grid, dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL(row_kernel<BAKRON_T_F16>, grid, dim3(NT), 0, s, a);
    BK_LAUNCH_CHECK("row_kernel");
    if (a.segs > 1) {
        const dim3 jg((unsigned)rows);
        if (type == BAKRON_T_F32)
            hipLaunchKernelGGL(join_kernel<BAKRON_T_F32>, jg, dim3(256), 0, s, a);
        else if (type == BAKRON_T_BF16)
            hipLaunchKernelGGL(join_kernel<BAKRON_T_BF16>, jg, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL(join_kernel<BAKRON_T_F16>, jg, dim3(256), 0, s, a);
        BK_LAUNCH_CHECK("join_kernel");
    }
    return BAKRON_OK;
}

extern "C" int32_t bakron_token_logprobs_grad(const void *logits, int32_t type, int64_t rows, int64_t vocab,
                                              int64_t ld, const int64_t *targets, const float *lse,
                                              const float *entropy, const float *g_logprob,
                                              const float *g_entropy, void *dlogits, int64_t ldd,
                                              int32_t *dev_status, void *stream_) {
    clear_error();
    BK_REQUIRE(logits && targets && lse && g_logprob && dlogits,
               "logits, targets, lse, g_logprob and dlogits must be non-NULL");
    BK_REQUIRE(!g_entropy || entropy, "g_entropy needs the forward pass's entropy");
    BK_REQUIRE(type == BAKRON_T_F32 || type == BAKRON_T_BF16 || type == BAKRON_T_F16, "bad type %d", type);
    BK_REQUIRE(rows >= 1 && rows <= MAX_ROWS && vocab >= 1 && vocab <= MAX_VOCAB,
               "bad sizes rows=%lld vocab=%lld", (long long)rows, (long long)vocab);
    BK_REQUIRE(ld >= vocab && ldd >= vocab && ld <= MAX_LD && ldd <= MAX_LD,
               "bad row strides ld=%lld ldd=%lld for a vocabulary of %lld", (long long)ld, (long long)ldd,
               (long long)vocab);
    BK_REQUIRE(((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) &
                (elem_size(type) - 1)) == 0,
               "logits or dlogits are misaligned for their type");
    const int64_t segs = (vocab + 8191) / 8192;
    BK_REQUIRE(rows * segs < (int64_t(1) << 31), "too many logits: rows=%lld vocab=%lld", (long long)rows,
               (long long)vocab);
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    const dim3 grid((unsigned)(rows * segs));
    const char *x = static_cast<const char *>(logits);
    char *dx = static_cast<char *>(dlogits);
    if (type == BAKRON_T_F32)
        hipLaunchKernelGGL(grad_kernel<BAKRON_T_F32>, grid, dim3(256), 0, s, x, vocab, ld, targets, lse,
                           entropy, g_logprob, g_entropy, dx, ldd, (int)segs, dev_status);
    else if (type == BAKRON_T_BF16)
        hipLaunchKernelGGL(grad_kernel<BAKRON_T_BF16>, grid, dim3(256), 0, s, x, vocab, ld, targets, lse,
                           entropy, g_logprob, g_entropy, dx, ldd, (int)segs, dev_status);
    else
        hipLaunchKernelGGL(grad_kernel<BAKRON_T_F16>, grid, dim3(256), 0, s, x, vocab, ld, targets, lse,
                           entropy, g_logprob, g_entropy, dx, ldd, (int)segs, dev_status);
    BK_LAUNCH_CHECK("grad_kernel");
    return BAKRON_OK;
}
