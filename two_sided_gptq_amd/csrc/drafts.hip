// drafts.hip -- bakron_verify_drafts: drafted tokens accepted or refused by the target's
// probabilities, from given random numbers.
//
// Draft d_i, drawn from q_i, is accepted where u_i q_i(d_i) < p_i(d_i).  At the first
// refusal the token is drawn from r = max(p_i - q_i, 0), after the last draft from p_i:
// the first x with r(0) + .. + r(x) > v sum r.  The tokens that come out are distributed
// as the target's own.  All of it is in 64 bits: products and differences of 32-bit numbers
// are exact there, and the sums' rounding (2^-53 of them) is far below the distance of
// a 24-bit v to the border of a token that 32-bit probabilities can express.
//
// Of all rows only the two at the first refusal are read, so the call is bound by HBM for
// many requests and by latency for few.  The row is cut into stretches, one a wave; their
// sums say in which the token lies, and that one is read again (from L2).  Sums are in a
// fixed order.
#include "common.hpp"
#include "elem.hpp"

namespace bakron {
namespace {

constexpr int NT = 1024;             // threads that finish a request
constexpr int WAVES = NT / 64;
constexpr int PART_WAVES = 4;        // waves of a workgroup that sums stretches only
constexpr int MAX_PARTS = 64;        // stretches of a row: a lane each
constexpr int MAX_DRAFTS = 64;
constexpr int64_t MAX_DIM = int64_t(1) << 24;

struct DraftArgs {
    const char *p, *q;       // q NULL: drafts without a distribution
    int64_t ldp, ldq;
    int vocab, drafts;
    const int64_t *tokens_in;
    const float *u, *v;
    int32_t *accepted;
    int64_t *tokens;
    int32_t *dev_status;
    int parts, length;       // stretches of a row and their elements
    double *part;            // [request][parts], where they are summed by a launch of their own
};

// What a request's token is drawn from, wave uniform.
struct Row {
    const char *p, *q;  // q: subtracted, or NULL
    int64_t at_p, at_q; // the rows' first elements
    int skip;           // a token of weight 0, or -1
};

struct Decision {
    int accepted;
    int64_t draft;  // in lane i: draft i
    bool refused, bad_index, nonfinite;
};

// Lane i holds draft i.  Drafts end at the first negative one.
template <int T>
__device__ __forceinline__ Decision decide(const DraftArgs &a, int64_t b) {
    const int i = threadIdx.x & 63;
    Decision d;
    d.draft = -1;
    bool good = false, odd = false, large = false;
    if (i < a.drafts) {
        d.draft = a.tokens_in[b * a.drafts + i];
        const float u = a.u[b * a.drafts + i];
        large = d.draft >= a.vocab;
        if (d.draft >= 0 && !large) {
            const float p = load1<T>(a.p, (b * (a.drafts + 1) + i) * a.ldp + d.draft);
            const float q = a.q ? load1<T>(a.q, (b * a.drafts + i) * a.ldq + d.draft) : 1.0f;
            good = (double)u * (double)q < (double)p;
            odd = !(__builtin_isfinite(p) && __builtin_isfinite(q));
        }
    }
    const uint64_t stop = ~__ballot(good), seen = stop & -stop;  // the first draft that is not accepted
    d.accepted = min(a.drafts, stop ? __ffsll((unsigned long long)stop) - 1 : 64);
    const uint64_t upto = seen | (seen - 1);
    d.refused = d.accepted < a.drafts && (__ballot(d.draft >= 0) & seen);
    d.bad_index = __ballot(large) & upto;
    d.nonfinite = __ballot(odd) & upto;
    return d;
}

template <int T>
__device__ __forceinline__ Row row_of(const DraftArgs &a, int64_t b, const Decision &d) {
    Row r;
    r.p = a.p, r.q = d.refused ? a.q : nullptr;
    r.at_p = (b * (a.drafts + 1) + d.accepted) * a.ldp;
    r.at_q = (b * a.drafts + d.accepted) * a.ldq;
    r.skip = -1;
    if (d.refused && !a.q) {
        const int64_t t = __shfl(d.draft, d.accepted);
        r.skip = t < a.vocab ? (int)t : -1;
    }
    return r;
}

// Weights of tokens x .. x + 7 of p (and q where the row has one).
__device__ __forceinline__ void weights_of(const Row &r, int x, const float *p, const float *q, double *w) {
    if (r.q) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double d = (double)p[e] - (double)q[e];
            w[e] = d < 0.0 ? 0.0 : d;  // a NaN stays one
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = p[e] < 0.0f || x + e == r.skip ? 0.0 : (double)p[e];
    }
}
// 0 from `left` on.
template <int T>
__device__ __forceinline__ void weights8(const Row &r, int x, int left, double *w) {
    float p[8], q[8] = {};
    load8<T>(r.p, r.at_p + x, left, p);
    if (r.q) load8<T>(r.q, r.at_q + x, left, q);
    weights_of(r, x, p, q, w);
}

__device__ __forceinline__ double sum8(const double *w) {
    return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    return s;
}

// The wave's sum of the weights of tokens [lo, hi): steps of 512, the loads of some on
// their way together.
template <int T>
__device__ __forceinline__ double stretch_sum(const Row &r, int lo, int hi) {
    constexpr int ES = Raw8<T>::ES, U = 8 / ES;  // in fp32 the registers hold 2
    double s = 0.0;
    const int lane = threadIdx.x & 63, steps = (hi - lo) / 512;
    const char *p = r.p + (r.at_p + lo + lane * 8) * ES, *q = r.q ? r.q + (r.at_q + lo + lane * 8) * ES : nullptr;
    for (int i = 0; i < steps; i += U) {
        Raw8<T> rp[U], rq[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i + k >= steps) break;
            __builtin_memcpy(rp[k].w, p + (i + k) * 512 * ES, 8 * ES);
            if (r.q) __builtin_memcpy(rq[k].w, q + (i + k) * 512 * ES, 8 * ES);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i + k >= steps) break;
            float x[8], y[8] = {};
            double w[8];
            unpack8<T>(rp[k].w, x);
            if (r.q) unpack8<T>(rq[k].w, y);
            weights_of(r, lo + (i + k) * 512 + lane * 8, x, y, w);
            s += sum8(w);
        }
    }
    const int x = lo + steps * 512 + lane * 8;
    if (x < hi) {
        double w[8];
        weights8<T>(r, x, hi - x, w);
        s += sum8(w);
    }
    return wave_sum(s);
}

template <int T>
__global__ __launch_bounds__(64 * PART_WAVES) void verify_part_kernel(DraftArgs a) {
    const int groups = a.parts / PART_WAVES;
    const int64_t b = blockIdx.x / groups;
    const int part = (int)(blockIdx.x - b * groups) * PART_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Decision d = decide<T>(a, b);
    const Row r = row_of<T>(a, b, d);
    const int lo = min(a.vocab, part * a.length), hi = min(a.vocab, lo + a.length);
    const double s = stretch_sum<T>(r, lo, hi);
    if ((threadIdx.x & 63) == 0) a.part[b * a.parts + part] = s;
}

// Inclusive sums of a value a lane.
__device__ __forceinline__ double wave_scan(double x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    return x;
}

// The first of 64 lanes whose sum up to it is above the target and whose own is not 0, or,
// where rounding leaves none, the last whose own is not 0.
__device__ __forceinline__ int pick(double upto, double own, double target) {
    const uint64_t some = __ballot(own > 0.0), hit = __ballot(upto > target) & some;
    if (hit) return __ffsll((unsigned long long)hit) - 1;
    return some ? 63 - __clzll((long long)some) : -1;
}

template <int T, bool SUMMED>
__global__ __launch_bounds__(NT) void verify_kernel(DraftArgs a) {
    __shared__ double sums[WAVES];
    __shared__ int found;
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Decision d = decide<T>(a, b);
    Row r = row_of<T>(a, b, d);
    const float vf = a.v[b];
    const double v = vf > 0.0f ? (double)vf : 0.0;  // a NaN counts as 0
    if (threadIdx.x == 0) found = -1;
    double own = 0.0, total;
    int length;
    if constexpr (SUMMED) {
        own = lane < a.parts ? a.part[b * a.parts + lane] : 0.0;
        length = a.length;
        total = __shfl(wave_scan(own), 63);
    }
    // sums by this workgroup: of the weights, and of p where no weight is left
    for (int pass = SUMMED ? 1 : 0;; ++pass) {
        if (pass != 1 || !SUMMED) {
            length = ((a.vocab + WAVES - 1) / WAVES + 7) / 8 * 8;
            const int lo = min(a.vocab, w * length), hi = min(a.vocab, lo + length);
            const double s = stretch_sum<T>(r, lo, hi);
            if (lane == 0) sums[w] = s;
            __syncthreads();
            own = lane < WAVES ? sums[lane] : 0.0;
            total = __shfl(wave_scan(own), 63);
            __syncthreads();
        }
        if (total != 0.0 || !(r.q || r.skip >= 0)) break;
        r.q = nullptr, r.skip = -1;
    }
    const bool finite = __builtin_isfinite(total);
    int token = -1;
    if (finite && total > 0.0) {
        double target = v * total;
        double upto = wave_scan(own);
        const int part = pick(upto, own, target);
        target -= part ? __shfl(upto, max(part - 1, 0)) : 0.0;
        // the stretch again, a few tokens a thread
        const int lo = part * length, hi = min(a.vocab, lo + length);
        const int each = (length + NT * 8 - 1) / (NT * 8) * 8;
        const int x0 = min(hi, lo + (int)threadIdx.x * each), x1 = min(hi, x0 + each);
        double mine = 0.0;
        for (int x = x0; x < x1; x += 8) {
            double e[8];
            weights8<T>(r, x, x1 - x, e);
#pragma unroll
            for (int k = 0; k < 8; ++k) mine += e[k];
        }
        const double inside = wave_scan(mine);
        if (lane == 63) sums[w] = inside;
        __syncthreads();
        const double of_wave = lane < WAVES ? sums[lane] : 0.0;
        const double waves = wave_scan(of_wave);
        const int in = pick(waves, of_wave, target);
        if (w == in) {
            target -= in ? __shfl(waves, max(in - 1, 0)) : 0.0;
            const int l = pick(inside, mine, target);
            double run = l ? __shfl(inside, max(l - 1, 0)) : 0.0;
            if (lane == l) {
                for (int x = x0; x < x1; x += 8) {
                    double e[8];
                    weights8<T>(r, x, x1 - x, e);
                    for (int k = 0; k < 8; ++k) {
                        if (run > target && token >= 0) break;
                        run += e[k];
                        if (e[k] > 0.0) token = x + k;
                    }
                }
                found = token;
            }
        }
        __syncthreads();
        token = found;
    }
    if ((int)threadIdx.x <= a.drafts) {
        const int64_t draft = d.draft;
        const int i = threadIdx.x;
        a.tokens[b * (a.drafts + 1) + i] = i < d.accepted ? draft : i == d.accepted ? token : -1;
        if (i == 0) a.accepted[b] = d.accepted;
    }
    if (threadIdx.x == 0 && a.dev_status) {
        const int32_t bits = (d.bad_index ? BAKRON_DEV_BAD_INDEX : 0) | (d.nonfinite || !finite ? BAKRON_DEV_NONFINITE : 0);
        if (bits) atomicOr(a.dev_status, bits);
    }
}

// Stretches that get a launch of their own, or 0.  A workgroup reads its two rows at about 1.2
// us for 16384 tokens, as long as there are no more than CUs; a launch more costs about 2 us
// and spreads that over the CUs that idle.  (One request: 32000 tokens 8.2 in two launches, 9.0
// in one, 16384: 8.2 and 7.9; 128 requests of 131072 fp32: 28.3 and 32.7, of 50001: 16.9 and
// 16.1.)  Stretches of 512 tokens at least, in about 1024 workgroups at most.
int parts_of(int64_t batch, int64_t vocab) {
    if (vocab * (256 - batch) < int64_t(6700000)) return 0;
    int parts = MAX_PARTS;
    while (parts > 8 && parts * batch > 4096) parts /= 2;
    while (parts > 4 && (int64_t)parts * 512 > vocab) parts /= 2;
    return parts;
}

template <int T>
void launch_verify(DraftArgs a, int64_t batch, hipStream_t s) {
    if (a.parts) {
        hipLaunchKernelGGL(verify_part_kernel<T>, dim3((unsigned)(batch * (a.parts / PART_WAVES))), dim3(64 * PART_WAVES), 0, s, a);
        hipLaunchKernelGGL((verify_kernel<T, true>), dim3((unsigned)batch), dim3(NT), 0, s, a);
    } else {
        hipLaunchKernelGGL((verify_kernel<T, false>), dim3((unsigned)batch), dim3(NT), 0, s, a);
    }
}

constexpr int64_t MAX_BATCH = int64_t(1) << 20;

bool sizes_ok(int64_t batch, int32_t drafts, int64_t vocab) {
    return batch >= 1 && batch <= MAX_BATCH && drafts >= 0 && drafts <= MAX_DRAFTS && vocab >= 1 && vocab <= MAX_DIM;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" size_t bakron_verify_drafts_workspace_size(int64_t batch, int32_t drafts, int64_t vocab) {
    if (!sizes_ok(batch, drafts, vocab)) return 0;
    const int parts = parts_of(batch, vocab);
    return parts ? align256((size_t)batch * parts * sizeof(double)) : 0;
}

extern "C" int32_t bakron_verify_drafts(const void *p, int64_t ldp, const void *q, int64_t ldq, int32_t type,
                                        int64_t batch, int32_t drafts, int64_t vocab, const int64_t *draft_tokens,
                                        const float *u, const float *v, int32_t *accepted, int64_t *tokens,
                                        int32_t *dev_status, void *ws, size_t ws_bytes, void *stream_) {
    clear_error();
    BK_REQUIRE(p && v && accepted && tokens, "p, v, accepted and tokens must be non-NULL");
    BK_REQUIRE(type == BAKRON_T_F32 || type == BAKRON_T_BF16 || type == BAKRON_T_F16, "bad type %d", type);
    BK_REQUIRE(sizes_ok(batch, drafts, vocab), "bad sizes batch=%lld drafts=%d vocab=%lld", (long long)batch, drafts,
               (long long)vocab);
    BK_REQUIRE(drafts == 0 || (draft_tokens && u), "draft_tokens and u must be non-NULL for drafts");
    BK_REQUIRE(ldp >= vocab && ldp <= MAX_LD, "bad row stride ldp=%lld for a vocabulary of %lld", (long long)ldp,
               (long long)vocab);
    BK_REQUIRE(!q || (ldq >= vocab && ldq <= MAX_LD), "bad row stride ldq=%lld for a vocabulary of %lld",
               (long long)ldq, (long long)vocab);
    BK_REQUIRE(((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & (elem_size(type) - 1)) == 0,
               "p or q is misaligned for its type");
    const size_t need = bakron_verify_drafts_workspace_size(batch, drafts, vocab);
    if (need && (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255))) {
        set_error("workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, ws_bytes);
        return BAKRON_ERR_WORKSPACE;
    }
    int32_t st = check_device();
    if (st != BAKRON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream_);
    DraftArgs a = {};
    a.p = static_cast<const char *>(p), a.q = drafts ? static_cast<const char *>(q) : nullptr;
    a.ldp = ldp, a.ldq = ldq, a.vocab = (int)vocab, a.drafts = drafts;
    a.tokens_in = draft_tokens, a.u = u, a.v = v, a.accepted = accepted, a.tokens = tokens, a.dev_status = dev_status;
    a.parts = parts_of(batch, vocab);
    a.length = a.parts ? (int)round_up((vocab + a.parts - 1) / a.parts, 8) : 0;
    a.part = static_cast<double *>(ws);
    if (type == BAKRON_T_F32)
        launch_verify<BAKRON_T_F32>(a, batch, s);
    else if (type == BAKRON_T_BF16)
        launch_verify<BAKRON_T_BF16>(a, batch, s);
    else
        launch_verify<BAKRON_T_F16>(a, batch, s);
    BK_LAUNCH_CHECK("draft verification");
    return BAKRON_OK;
}
