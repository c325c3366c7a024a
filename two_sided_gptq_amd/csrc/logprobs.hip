// logprobs.hip -- bakron_token_logprobs and its gradient.
//
// For a row of logits x over a vocabulary of V tokens, with m = max x,
// s = sum e^(x - m) and t = sum e^(x - m) (x - m):
//   lse = m + log s,  log p_j = (x_j - m) - log s,  H = -sum p log p = log s - t / s.
// (x_j - lse would lose log s where |m| is large: in a row of the type's lowest value
// every token would get the probability 1.)  One pass over the row keeps (m, s, t) and
// rescales the two sums where the maximum grows; sums and statistics are fp32.
//
// Alternatives (the k largest, equal values by lowest index).  Each thread reads
// chunks of consecutive elements and leaves each chunk's maximum.  An element of the k
// largest lies in one of the k chunks that come first by (maximum, lowest chunk): any
// other chunk has k chunks before it, each with an element that is larger, or equal at
// a lower index.  So after the pass only k chunks are read again (from L2).  The
// selections are by counting: the rank of a key among a short list is the number of
// keys above it.
//
// Many rows: a workgroup takes a row.  Few rows: each is split over workgroups that
// leave their statistics and chunk maxima in the workspace, and a second launch joins
// the statistics in a fixed order and selects.
#include "common.hpp"
#include "elem.hpp"

namespace bakron {
namespace {

constexpr int NT = 512;      // threads that take a row, or join one
constexpr int NTS = 256;     // threads that take a part of a row
constexpr int CE = 16;       // elements that a thread reads at once
constexpr int CHUNKS = 8192; // chunks of a row at most: 32 KB of maxima in LDS
constexpr int KMAX = 64;
constexpr int CAP = 1024;    // candidates held in LDS

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
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, false);
    return ((uint64_t)hi << 32) | lo;
}
// The largest of 8 neighbouring lanes, in each of them.
__device__ __forceinline__ uint64_t max_of_8(uint64_t v) {
    v = max64(v, dpp64<0xb1>(v));   // quad_perm 1,0,3,2
    v = max64(v, dpp64<0x4e>(v));   // quad_perm 2,3,0,1
    return max64(v, dpp64<0x141>(v));  // row_half_mirror: the other four
}

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

// How many of list[0, n) are above key; list[n] is 0 and the list 16-byte aligned.
__device__ __forceinline__ int rank_of(const uint64_t *list, int n, uint64_t key) {
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; j += 2) {
        const ulong2 two = *reinterpret_cast<const ulong2 *>(list + j);
        rank += (two.x > key) + (two.y > key);
    }
    return rank;
}

// The k best of list[0, n) (distinct keys, n <= CAP; 0 entries are none) into
// out[0, k) in order; places without a key get 0.
__device__ __forceinline__ void rank_select(uint64_t *list, int n, uint64_t *out, int k) {
    for (int i = threadIdx.x; i < k; i += blockDim.x) out[i] = 0;
    if (threadIdx.x == 0) list[n] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint64_t key = list[i];
        const int rank = rank_of(list, n, key);
        if (rank < k && key) out[rank] = key;
    }
    __syncthreads();
}

struct RowArgs {
    const char *x;
    int64_t rows, vocab, ld;
    const int64_t *targets;
    int k, runs;         // a chunk is `runs` times CE elements
    int chunks;          // of a row
    int segs, per_seg;   // parts of a row, chunks of a part
    float *logprob, *lse, *entropy, *top_logprob;
    int64_t *top_ids;
    int32_t *dev_status;
    Stats *part;   // [rows][segs]
    float *maxima; // [rows][chunks]
};

// A row's target and its logit; asked for before the statistics are known, as the two
// loads depend on each other.
struct Target {
    int64_t t;
    float x;
};
template <int T>
__device__ __forceinline__ Target target_of(const RowArgs &a, int64_t row) {
    Target r = {a.targets[row], 0.0f};
    if (r.t >= 0 && r.t < a.vocab) r.x = load1<T>(a.x, row * a.ld + r.t);
    return r;
}

// What log probabilities are taken from: log p = (x - m) - logs.  logs is -inf in a row
// without a distribution and NaN in one that holds a NaN or +inf.
struct Norm {
    float m, logs;
    __device__ __forceinline__ float operator()(float x) const { return logs == -INFINITY ? -INFINITY : (x - m) - logs; }
};

// What a row's statistics give; one thread.
__device__ __forceinline__ Norm finish_row(const RowArgs &a, int64_t row, Stats st, Target target) {
    const bool none = st.s == 0.0f;                    // every logit is -inf
    const bool bad = st.s != st.s || st.m > 3.4028235e38f;  // a NaN or +inf
    const float nan = __uint_as_float(0x7fc00000u);
    const Norm norm = {st.m, bad ? nan : none ? -INFINITY : __logf(st.s)};
    float lse = none ? -INFINITY : st.m + norm.logs;
    float ent = none ? 0.0f : norm.logs - st.t / st.s;
    if (bad) lse = ent = nan;
    int32_t flag = bad ? BAKRON_DEV_NONFINITE : 0;
    a.lse[row] = lse;
    a.entropy[row] = ent;
    float lp = 0.0f;
    if (target.t >= a.vocab) {
        lp = nan;
        flag |= BAKRON_DEV_BAD_INDEX;
    } else if (target.t >= 0) {
        lp = norm(target.x);
    }
    a.logprob[row] = lp;
    if (flag && a.dev_status) atomicOr(a.dev_status, flag);
    return norm;
}

__device__ __forceinline__ void write_top(const RowArgs &a, int64_t row, const uint64_t *best, Norm norm) {
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
        const uint64_t key = best[i];
        a.top_logprob[row * a.k + i] = norm(unorder((uint32_t)(key >> 32)));
        a.top_ids[row * a.k + i] = (int64_t)(uint32_t)~(uint32_t)key;
    }
}

// Statistics of a thread's chunks c0 + tid, + threads, .. below c1, with their maxima.
template <int T, int THREADS>
__device__ __forceinline__ Stats take_chunks(const RowArgs &a, int64_t base, int c0, int c1, float *maxima) {
    Stats st = {-3.4028235e38f, 0.0f, 0.0f};
    for (int c = c0 + threadIdx.x; c < c1; c += THREADS) {
        float top = -INFINITY;
        for (int u = 0; u < a.runs; ++u) {
            const int64_t e = ((int64_t)c * a.runs + u) * CE;
            float x[CE];
            if (e + CE <= a.vocab) {
                load8<T>(a.x, base + e, 8, x);
                load8<T>(a.x, base + e + 8, 8, x + 8);
            } else {
#pragma unroll
                for (int q = 0; q < CE; ++q) x[q] = e + q < a.vocab ? load1<T>(a.x, base + e + q) : -INFINITY;
            }
            float cm = x[0];
#pragma unroll
            for (int q = 1; q < CE; ++q) cm = fmaxf(cm, x[q]);
            top = fmaxf(top, cm);
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
        if (maxima) maxima[c] = top;
    }
    return st;
}

// Statistics of the whole workgroup, in its thread 0.
template <int THREADS>
__device__ __forceinline__ Stats block_stats(Stats st, Stats *wave_part) {
    st = wave_stats(st);
    if ((threadIdx.x & 63) == 0) wave_part[threadIdx.x >> 6] = st;
    __syncthreads();
    if (threadIdx.x == 0) {
        st = wave_part[0];
        for (int i = 1; i < THREADS / 64; ++i) st = merge(st, wave_part[i]);
    }
    return st;
}

struct TopSpace {
    float cmax[CHUNKS];
    __align__(16) uint64_t list[CAP + 2];
    uint64_t best[KMAX], bound;
    int count;
};

// The k best elements of a row into best[0, k), from its chunks' maxima.  NT threads.
template <int T>
__device__ void select_top(const RowArgs &a, int64_t base, TopSpace &s) {
    const int k = a.k, tid = threadIdx.x;
    // a lower bound of the k-th best chunk: the k-th of 64 groups' best chunks
    uint64_t grp = 0;
    for (int c = tid; c < a.chunks; c += NT) grp = max64(grp, key_of(s.cmax[c], (uint32_t)c));
    grp = max_of_8(grp);
    if ((tid & 7) == 0) s.list[tid >> 3] = grp;
    if (tid == 0) s.bound = 0, s.count = 0;
    __syncthreads();
    if (tid < 64) {
        const uint64_t key = s.list[tid];
        if (rank_of(s.list, 64, key) == k - 1 && key) s.bound = key;  // keys other than 0 are distinct
    }
    __syncthreads();
    const uint64_t bound = s.bound;
    if (grp >= bound && grp)
        for (int c = tid; c < a.chunks; c += NT) {
            const uint64_t key = key_of(s.cmax[c], (uint32_t)c);
            if (key >= bound) {
                const int at = atomicAdd(&s.count, 1);
                if (at < CAP) s.list[at] = key;
            }
        }
    __syncthreads();
    const int n = s.count;
    if (n <= CAP) {
        rank_select(s.list, n, s.best, k);
    } else {
        // far more chunks above the bound than usual: one by one
        uint64_t last = ~0ull;
        for (int i = 0; i < k; ++i) {
            uint64_t top = 0;
            for (int c = tid; c < a.chunks; c += NT) {
                const uint64_t key = key_of(s.cmax[c], (uint32_t)c);
                if (key < last) top = max64(top, key);
            }
            top = max_of_8(top);
            if ((tid & 7) == 0) s.list[tid >> 3] = top;
            __syncthreads();
            for (int j = 0; j < NT / 8; ++j) top = max64(top, s.list[j]);
            if (tid == 0) s.best[i] = top;
            last = top;
            __syncthreads();
        }
    }
    // of longer chunks, the runs of CE elements that reach the k-th chunk's maximum
    if (a.runs > 1) {
        const uint64_t floor = s.best[k - 1] >> 32;
        if (tid == 0) s.count = 0;
        __syncthreads();
        for (int i = tid; i < k * a.runs; i += NT) {  // at most CAP
            const uint64_t ck = s.best[i / a.runs];
            const uint32_t r = ~(uint32_t)ck * (uint32_t)a.runs + (uint32_t)(i % a.runs);
            const int64_t e = (int64_t)r * CE;
            if (!ck || e >= a.vocab) continue;
            float top = load1<T>(a.x, base + e);
            for (int q = 1; q < CE && e + q < a.vocab; ++q) top = fmaxf(top, load1<T>(a.x, base + e + q));
            const uint64_t key = key_of(top, r);
            if ((key >> 32) >= floor) s.list[atomicAdd(&s.count, 1)] = key;
        }
        __syncthreads();
        rank_select(s.list, s.count, s.best, k);
    }
    // the elements of the k runs that reach the k-th one's maximum
    const uint64_t floor = s.best[k - 1] >> 32;
    if (tid == 0) s.count = 0;
    __syncthreads();
    for (int i = tid; i < k * CE; i += NT) {  // at most CAP
        const uint64_t ck = s.best[i / CE];
        const int64_t e = (int64_t)(uint32_t)~(uint32_t)ck * CE + i % CE;
        if (ck && e < a.vocab) {
            const uint64_t key = key_of(load1<T>(a.x, base + e), (uint32_t)e);
            if ((key >> 32) >= floor) s.list[atomicAdd(&s.count, 1)] = key;
        }
    }
    __syncthreads();
    rank_select(s.list, s.count, s.best, k);
}

// One row.
template <int T>
__global__ __launch_bounds__(NT) void row_kernel(RowArgs a) {
    __shared__ TopSpace top;
    __shared__ Stats wave_part[NT / 64];
    __shared__ Norm norm;
    const int64_t row = blockIdx.x, base = row * a.ld;
    Target target = {-1, 0.0f};
    if (threadIdx.x == 0) target = target_of<T>(a, row);
    Stats st = take_chunks<T, NT>(a, base, 0, a.chunks, a.k ? top.cmax : nullptr);
    st = block_stats<NT>(st, wave_part);
    if (threadIdx.x == 0) norm = finish_row(a, row, st, target);
    if (a.k == 0) return;
    __syncthreads();
    select_top<T>(a, base, top);
    write_top(a, row, top.best, norm);
}

// One part of a row.
template <int T>
__global__ __launch_bounds__(NTS) void part_kernel(RowArgs a) {
    __shared__ Stats wave_part[NTS / 64];
    const int64_t row = blockIdx.x / a.segs;
    const int sg = (int)(blockIdx.x - row * a.segs);
    const int c0 = sg * a.per_seg, c1 = min(a.chunks, c0 + a.per_seg);
    Stats st = take_chunks<T, NTS>(a, row * a.ld, c0, c1, a.k ? a.maxima + row * a.chunks : nullptr);
    st = block_stats<NTS>(st, wave_part);
    if (threadIdx.x == 0) a.part[blockIdx.x] = st;
}

// Joins a row's parts: statistics in a fixed order, and the selection.
template <int T>
__global__ __launch_bounds__(NT) void join_kernel(RowArgs a) {
    __shared__ TopSpace top;
    __shared__ Norm norm;
    const int64_t row = blockIdx.x;
    Target target = {-1, 0.0f};
    if (threadIdx.x == 0) target = target_of<T>(a, row);
    if (a.k)
#pragma unroll 8
        for (int c = threadIdx.x; c < a.chunks; c += NT) top.cmax[c] = a.maxima[row * a.chunks + c];
    if (threadIdx.x < 64) {
        Stats st = {-3.4028235e38f, 0.0f, 0.0f};
        for (int i = threadIdx.x; i < a.segs; i += 64) st = merge(st, a.part[row * a.segs + i]);
        st = wave_stats(st);
        if (threadIdx.x == 0) norm = finish_row(a, row, st, target);
    }
    if (a.k == 0) return;
    __syncthreads();
    select_top<T>(a, row * a.ld, top);
    write_top(a, row, top.best, norm);
}

// d logits = -p (g + g_H (log p + H)), and g more at the target.  log p = x - lse: of the
// row's statistics the backward pass has no more.
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

// How a launch is laid out.  A workgroup to a row where there are rows for every CU,
// or where a row is short; else parts of no less than 4096 elements, up to about 1024
// of them (8 rows of 131072 bf16 logits, k = 20: 14 us in 32 parts a row).
void layout(RowArgs &a) {
    a.runs = (int)((a.vocab + (int64_t)CHUNKS * CE - 1) / ((int64_t)CHUNKS * CE));
    a.chunks = (int)((a.vocab + a.runs * CE - 1) / (a.runs * CE));
    int64_t segs = a.rows >= 512 ? 1 : (1024 + a.rows - 1) / a.rows;
    if (segs > a.chunks / NTS) segs = a.chunks / NTS;
    if (segs < 1) segs = 1;
    a.per_seg = (int)round_up((a.chunks + segs - 1) / segs, NTS);
    a.segs = (a.chunks + a.per_seg - 1) / a.per_seg;
}

template <int T>
void launch_rows(const RowArgs &all, hipStream_t s) {
    RowArgs a = all;
    if (a.segs == 1) {
        constexpr int64_t most = LAUNCH_THREADS / NT;
        for (int64_t left = a.rows; left > 0; left -= most) {
            a.rows = left < most ? left : most;
            hipLaunchKernelGGL(row_kernel<T>, dim3((unsigned)a.rows), dim3(NT), 0, s, a);
            a.x += a.rows * a.ld * elem_size(T), a.targets += a.rows;
            a.logprob += a.rows, a.lse += a.rows, a.entropy += a.rows;
            if (a.k) a.top_logprob += a.rows * a.k, a.top_ids += a.rows * a.k;
        }
        return;
    }
    hipLaunchKernelGGL(part_kernel<T>, dim3((unsigned)(a.rows * a.segs)), dim3(NTS), 0, s, a);
    hipLaunchKernelGGL(join_kernel<T>, dim3((unsigned)a.rows), dim3(NT), 0, s, a);
}

struct GradArgs {
    const char *x;
    int64_t rows, vocab, ld;
    const int64_t *targets;
    const float *lse, *entropy, *g_logprob, *g_entropy;
    char *dx;
    int64_t ldd;
    int32_t *dev_status;
};

template <int T>
void launch_grad(const GradArgs &a, hipStream_t s) {
    const int64_t segs = (a.vocab + 8191) / 8192, most = LAUNCH_THREADS / 256 / segs;  // rows of a launch
    for (int64_t r = 0; r < a.rows; r += most) {
        const int64_t rows = a.rows - r < most ? a.rows - r : most;
        hipLaunchKernelGGL(grad_kernel<T>, dim3((unsigned)(rows * segs)), dim3(256), 0, s,
                           a.x + r * a.ld * elem_size(T), a.vocab, a.ld, a.targets + r, a.lse + r,
                           a.entropy ? a.entropy + r : nullptr, a.g_logprob + r, a.g_entropy ? a.g_entropy + r : nullptr,
                           a.dx + r * a.ldd * elem_size(T), a.ldd, (int)segs, a.dev_status);
    }
}

constexpr int64_t MAX_VOCAB = (int64_t)CHUNKS * CE * (CAP / KMAX);  // 2^21
constexpr int64_t MAX_ROWS = int64_t(1) << 24;

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" size_t bakron_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t k) {
    if (rows < 1 || rows > MAX_ROWS || vocab < 1 || vocab > MAX_VOCAB || k < 0 || k > KMAX || k > vocab) return 0;
    RowArgs a = {};
    a.rows = rows, a.vocab = vocab;
    layout(a);
    if (a.segs == 1) return 0;
    return align256(rows * a.segs * sizeof(Stats)) + (k ? align256(rows * a.chunks * sizeof(float)) : 0);
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
    a.rows = rows, a.vocab = vocab;
    layout(a);
    const size_t need = bakron_token_logprobs_workspace_size(rows, vocab, k);
    if (need && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255))) {
        set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, ws_bytes);
        return BAKRON_ERR_WORKSPACE;
    }
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    a.x = static_cast<const char *>(logits);
    a.ld = ld, a.targets = targets, a.k = k;
    a.logprob = logprob, a.lse = lse, a.entropy = entropy;
    a.top_logprob = top_logprob, a.top_ids = top_ids, a.dev_status = dev_status;
    if (a.segs > 1) {
        Carver c(ws);
        a.part = c.take<Stats>(rows * a.segs);
        a.maxima = c.take<float>(k ? rows * a.chunks : 0);
    }
    if (type == BAKRON_T_F32)
        launch_rows<BAKRON_T_F32>(a, s);
    else if (type == BAKRON_T_BF16)
        launch_rows<BAKRON_T_BF16>(a, s);
    else
        launch_rows<BAKRON_T_F16>(a, s);
    BK_LAUNCH_CHECK("token log probabilities");
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
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    const GradArgs a = {static_cast<const char *>(logits), rows, vocab, ld, targets, lse, entropy, g_logprob, g_entropy,
                        static_cast<char *>(dlogits), ldd, dev_status};
    if (type == BAKRON_T_F32)
        launch_grad<BAKRON_T_F32>(a, s);
    else if (type == BAKRON_T_BF16)
        launch_grad<BAKRON_T_BF16>(a, s);
    else
        launch_grad<BAKRON_T_F16>(a, s);
    BK_LAUNCH_CHECK("grad_kernel");
    return BAKRON_OK;
}
