// sample.cu -- a token from each row of logits, drawn with given random numbers under temperature,
// top-k, top-p and min-p (mnb_sample).
//
// The tokens of a row are ordered by falling logit, equal ones by rising id; every limit keeps a
// prefix of that order, and the drawn token is the first whose cumulative weight passes u times
// the kept weight.  So three places in one order are wanted, each "the first at which a running sum
// reaches a target", and nothing has to be sorted: FP16 logits have few distinct values,
// and equal ones weigh the same.  A histogram over the 16-bit order of the logits, from
// the largest down (the window), gives counts and lowest ids; with one weight a distinct value, taken to
// 2^-40, the sums are those that 64-bit arithmetic gives.
//
//   look 1   the row's maximum, and how far down the window has to reach: to the n-th largest of
//            the threads' maxima, so at least n logits are in it (or to the histogram's end)
//   look 2   the histogram; what lies below the window enters as a sum in FP32 with a bound
//            of its error.  With a top-k it is not needed.
// Where the two ends of that bound give the same token, it is the token.  Else the window is widened
// to all of the histogram's places, and after that the row is gone through window by window to its end,
// which leaves nothing inexact.  A drawn value that several tokens share takes one more
// look for the id.
//
// A cluster of up to eight CTAs takes a row; the histogram is in its first one's shared memory, where the
// others add with remote atomics (integers: their order does not matter).
#include <cuda_fp16.h>

#include "common.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 24;
constexpr int kBins = 4096;              // places of the window
constexpr int kMaxWindows = 65536 / kBins + 2;
constexpr uint32_t kLowest = 0x0400;     // order of -65504, the lowest logit that can be drawn
constexpr uint32_t kInfinite = 0xFC00;   // order of +infinity; NaN lies above
constexpr int kAll = INT32_MAX;          // no limit
constexpr int kBeyond = kAll - 1;        // a limit somewhere below the window

struct SampleArgs {
    const __half* logits;
    int64_t rows, row_stride;
    int vocab, cluster;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int64_t* token;
    float* logprob;
};

// 2^(j / 64), j = -32 .. 32
__constant__ double kRoots[65] = {
    0x1.6a09e667f3bcdp-1, 0x1.6dfb23c651a2fp-1, 0x1.71f75e8ec5f74p-1, 0x1.75feb564267c9p-1,
    0x1.7a11473eb0187p-1, 0x1.7e2f336cf4e62p-1, 0x1.82589994cce13p-1, 0x1.868d99b4492edp-1,
    0x1.8ace5422aa0dbp-1, 0x1.8f1ae99157736p-1, 0x1.93737b0cdc5e5p-1, 0x1.97d829fde4e50p-1,
    0x1.9c49182a3f090p-1, 0x1.a0c667b5de565p-1, 0x1.a5503b23e255dp-1, 0x1.a9e6b5579fdbfp-1,
    0x1.ae89f995ad3adp-1, 0x1.b33a2b84f15fbp-1, 0x1.b7f76f2fb5e47p-1, 0x1.bcc1e904bc1d2p-1,
    0x1.c199bdd85529cp-1, 0x1.c67f12e57d14bp-1, 0x1.cb720dcef9069p-1, 0x1.d072d4a07897cp-1,
    0x1.d5818dcfba487p-1, 0x1.da9e603db3285p-1, 0x1.dfc97337b9b5fp-1, 0x1.e502ee78b3ff6p-1,
    0x1.ea4afa2a490dap-1, 0x1.efa1bee615a27p-1, 0x1.f50765b6e4540p-1, 0x1.fa7c1819e90d8p-1,
    0x1.0000000000000p+0, 0x1.02c9a3e778061p+0, 0x1.059b0d3158574p+0, 0x1.0874518759bc8p+0,
    0x1.0b5586cf9890fp+0, 0x1.0e3ec32d3d1a2p+0, 0x1.11301d0125b51p+0, 0x1.1429aaea92de0p+0,
    0x1.172b83c7d517bp+0, 0x1.1a35beb6fcb75p+0, 0x1.1d4873168b9aap+0, 0x1.2063b88628cd6p+0,
    0x1.2387a6e756238p+0, 0x1.26b4565e27cddp+0, 0x1.29e9df51fdee1p+0, 0x1.2d285a6e4030bp+0,
    0x1.306fe0a31b715p+0, 0x1.33c08b26416ffp+0, 0x1.371a7373aa9cbp+0, 0x1.3a7db34e59ff7p+0,
    0x1.3dea64c123422p+0, 0x1.4160a21f72e2ap+0, 0x1.44e086061892dp+0, 0x1.486a2b5c13cd0p+0,
    0x1.4bfdad5362a27p+0, 0x1.4f9b2769d2ca7p+0, 0x1.5342b569d4f82p+0, 0x1.56f4736b527dap+0,
    0x1.5ab07dd485429p+0, 0x1.5e76f15ad2148p+0, 0x1.6247eb03a5585p+0, 0x1.6623882552225p+0,
    0x1.6a09e667f3bcdp+0,
};

// FP16 bits as an unsigned value in the same order: -0 as +0, NaN the largest.
__device__ __forceinline__ uint32_t order16(uint32_t h) {
    h = h == 0x8000u ? 0u : h;
    h = (h & 0x7FFFu) > 0x7C00u ? 0x7FFFu : h;
    return (h & 0x8000u) ? (~h & 0xFFFFu) : (h | 0x8000u);
}

__device__ __forceinline__ uint32_t unorder16(uint32_t o) { return (o & 0x8000u) ? (o & 0x7FFFu) : (~o & 0xFFFFu); }

__device__ __forceinline__ float value_of(uint32_t o) {
    return __half2float(__ushort_as_half((unsigned short)unorder16(o)));
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a row's weights are taken with: 2^(c (logit - top)), c = log2(e) / temperature.
struct Scale {
    float top, c, c_low;  // c in two words
};

// log2 of the weight of a logit, in two words.
__device__ __forceinline__ float2 power_of(const Scale& k, float logit) {
    // the difference is exact in two words
    const float s = __fsub_rn(logit, k.top), b = __fsub_rn(s, logit);
    const float e = __fsub_rn(__fsub_rn(logit, __fsub_rn(s, b)), __fadd_rn(k.top, b));
    const float p = __fmul_rn(s, k.c);
    return make_float2(p, __fmaf_rn(s, k.c, -p) + __fmaf_rn(s, k.c_low, __fmul_rn(e, k.c)));
}

// 2^(p.x + p.y) to 2^-40: 2^n times a root of two from a table times the exponential series of what is left
// (at most ln 2 / 128), whose first term is kept in two words.
__device__ __forceinline__ double exp2_of(float2 p) {
    if (!(p.x > -1000.f)) return 0.0;
    const float n = rintf(p.x), f = p.x - n;  // exact
    const float j = rintf(f * 64.f), g = __fmaf_rn(j, -0.015625f, f);  // exact
    const float h = __fmul_rn(g, 0.6931471824645996f);
    const float l = __fmaf_rn(g, 0.6931471824645996f, -h) + __fmaf_rn(g, -1.9046542121259336e-09f, __fmul_rn(p.y, 0.6931471824645996f));
    const float z = h + l;
    const float q = z * z * (0.5f + z * (0.16666667f + z * (0.041666668f + z * 0.008333334f)));
    const double r = kRoots[(int)j + 32] * (1.0 + (double)h + (double)(l + q));
    return r * __longlong_as_double((long long)((int)n + 1023) << 52);
}

__device__ __forceinline__ double weight_of(const Scale& k, uint32_t order) {
    return exp2_of(power_of(k, value_of(order)));
}

// The lowest order of a window from `high` down.
__device__ __forceinline__ uint32_t window_low(uint32_t high) {
    return high >= kLowest + kBins ? high - (kBins - 1) : kLowest;
}

// ---- cluster ------------------------------------------------------------------

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void add_cluster(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void min_cluster(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- shared state ---------------------------------------------------------------

enum { kDone, kWindow, kTie, kScan };

struct Command {
    uint32_t op;
    uint32_t high, low;  // kWindow: the orders from `high` down to `low`
    uint32_t rest;       // kWindow: whether what lies below is summed
    uint32_t order;      // kTie, kScan: the order looked for
    uint32_t skip;       // kScan: of its tokens in this CTA's warp, the one after so many ...
    uint32_t who;        // ... in this warp of the cluster
};

struct Found {      // a place in the order
    int n;          // tokens up to and with it (0: not in the window)
    uint32_t order; // its logit
    int tie;        // tokens of that logit before it
    double sum;     // weight up to and with it
    double weight;  // its own
};

struct __align__(16) SampleShared {
    uint32_t count[kBins];
    uint32_t lowest[kBins];
    double warp_sum[kWarps];
    int warp_count[kWarps];
    double rest[kMaxCluster];           // first CTA: every CTA's sum below the window
    uint32_t below[kMaxCluster];        // ... and the largest order there
    uint32_t top[kMaxCluster], reach[kMaxCluster];  // all CTAs: every CTA's largest order, its n-th largest thread
    uint32_t ties[kMaxCluster * kWarps];
    uint32_t warp_word[kWarps];
    Command cmd;
    Found found[4];                     // the k-th or last kept, two places by weight, min-p's
    double win_sum[kMaxWindows];        // the search to the end: weight and tokens above each window,
    int win_count[kMaxWindows];         // and its bounds
    uint32_t win_high[kMaxWindows], win_low[kMaxWindows];
};

// A CTA's slice of a row: 16-byte pieces, and what is left at the row's ends.
struct Slice {
    const __half* row;
    int head, tail, pieces, vocab;  // logits before and behind the row's pieces
    int p0, p1;                     // pieces of this CTA
    bool first, last;
};

// The piece whose logits are those at the row's start (which = 0) or end, filled up with -infinity; *id: the token
// that its first place would be.
__device__ __forceinline__ uint4 edge_piece(const Slice& s, int which, int* id) {
    uint32_t w[4];
    *id = which ? s.head + s.pieces * 8 : s.head - 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = *id + i;
        const bool there = which ? at < s.vocab : at >= 0;
        const uint32_t h = there ? __half_as_ushort(s.row[there ? at : 0]) : 0xFC00u;
        w[i >> 1] = i & 1 ? w[i >> 1] | h << 16 : h;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// f(piece, id of its first logit) for all of the slice, several pieces in flight a thread.
template <typename F>
__device__ __forceinline__ void each_piece(const Slice& s, F f) {
    constexpr int kU = 4;
    const int tid = threadIdx.x;
    const uint4* p = reinterpret_cast<const uint4*>(s.row + s.head);
    int i = s.p0 + tid;
    for (; i + (kU - 1) * kThreads < s.p1; i += kU * kThreads) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = p[i + u * kThreads];
#pragma unroll
        for (int u = 0; u < kU; ++u) f(v[u], s.head + (i + u * kThreads) * 8);
    }
    for (; i < s.p1; i += kThreads) f(p[i], s.head + i * 8);
    int id;
    if (s.first && s.head && tid == kThreads - 1) {
        const uint4 v = edge_piece(s, 0, &id);
        f(v, id);
    }
    if (s.last && s.tail && tid == kThreads - 2) {
        const uint4 v = edge_piece(s, 1, &id);
        f(v, id);
    }
}

__device__ __forceinline__ uint32_t half_at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? w >> 16 : w & 0xFFFFu;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

__device__ __forceinline__ __half2 max_nan2(__half2 a, __half2 b) { return __hmax2_nan(a, b); }

__device__ __forceinline__ uint32_t block_max(SampleShared& sh, uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) sh.warp_word[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, sh.warp_word[threadIdx.x & (kWarps - 1)]);
}

// ---- the first CTA's search in the window -----------------------------------------

// A thread's bins with what lies before them.
struct Bins {
    int lo, hi;       // bins [lo, hi) of the window, largest logits first
    int before, n;    // tokens before them, and in them
    double above, end;  // the weight before them, and with them
};

// Sums of every thread's bins; *count, *sum: tokens and weight up to the window's end.
__device__ Bins window_bins(SampleShared& sh, const Scale& k, uint32_t high, uint32_t low, int before, double above,
                            int* count, double* sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = (int)(high - low) + 1, own = (bins + kThreads - 1) / kThreads;
    Bins b;
    b.lo = min(tid * own, bins);
    b.hi = min(b.lo + own, bins);
    b.n = 0;
    double w = 0.0;
    for (int i = b.lo; i < b.hi; ++i)
        if (sh.count[i]) {
            b.n += (int)sh.count[i];
            w += (double)sh.count[i] * weight_of(k, high - i);
        }
    int n = b.n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int pn = __shfl_up_sync(0xffffffffu, n, d);
        const double pw = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) n += pn, w += pw;
    }
    if (lane == 31) sh.warp_count[warp] = n, sh.warp_sum[warp] = w;
    __syncthreads();
    int wn = before, tn = before;
    double ws = above, ts = above;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i == warp) wn = tn, ws = ts;
        tn += sh.warp_count[i];
        ts += sh.warp_sum[i];
    }
    b.before = wn + n - b.n;
    const double pw = __shfl_up_sync(0xffffffffu, w, 1);
    b.above = ws + (lane ? pw : 0.0);  // the same sums as the end of the thread before
    b.end = ws + w;
    *count = tn;
    *sum = ts;
    return b;
}

// Walks a thread's bins to the first place where `stop(tokens, weight)` with the bin's tokens holds; there
// take(tokens before, weight before, bin's tokens, weight of one) gives how many of the bin's tokens, 1 ..
template <typename Stop, typename Take>
__device__ __forceinline__ void walk(const SampleShared& sh, const Scale& k, const Bins& b, uint32_t high, Found* out,
                                     Stop stop, Take take) {
    int n = b.before;
    double w = b.above;
    Found f = {};
    for (int i = b.lo; i < b.hi; ++i) {
        const int c = (int)sh.count[i];
        if (!c) continue;
        const double one = weight_of(k, high - i), to = w + (double)c * one;
        const bool here = stop(n + c, to);
        const int m = here ? take(n, w, c, one) : c;
        f = {n + m, high - (uint32_t)i, m - 1, w + (double)m * one, one};  // the last one where none stops
        if (here) break;
        n += c;
        w = to;
    }
    *out = f;
}

// The n-th token.
__device__ __forceinline__ void find_count(SampleShared& sh, const Scale& k, const Bins& b, uint32_t high, int n,
                                           Found* out) {
    if (b.n && b.before < n && n <= b.before + b.n)
        walk(sh, k, b, high, out, [&](int to, double) { return to >= n; },
             [&](int from, double, int, double) { return n - from; });
}

// The first token at which the weight reaches (or, PASS, passes) the target.
template <bool PASS>
__device__ __forceinline__ void find_weight(SampleShared& sh, const Scale& k, const Bins& b, uint32_t high, int first,
                                            double target, Found* out) {
    const bool mine = PASS ? b.above <= target && target < b.end
                           : (b.above < target || b.before == first) && target <= b.end;
    if (b.n && mine)
        walk(sh, k, b, high, out, [&](int, double to) { return PASS ? to > target : to >= target; },
             [&](int, double from, int c, double one) {
                 const double m = (target - from) / one;
                 const double i = PASS ? floor(m) + 1.0 : ceil(m);
                 return (int)fmin(fmax(i, 1.0), (double)c);
             });
}

// What a row asks for.
struct Wish {
    int k;         // kAll: no limit
    double p, m;   // 1 and above: no top-p; 0: no min-p
    double u;      // 1 and above: the last
};

// The last token of at least min_p times the largest weight; n = kAll where the window's last logit still is, and
// there is more below.
__device__ __forceinline__ void find_min_p(SampleShared& sh, const Scale& k, const Bins& b, uint32_t high, uint32_t low,
                                           bool more, double m, Found* out) {
    // the bin whose logits are kept and whose next bin's are not: one thread's, empty or not
    if (threadIdx.x == 0) {
        if (more && weight_of(k, low) >= m) *out = {kAll, 0, 0, 0.0, 0.0};
    }
    int n = b.before;
    double w = b.above;
    Found f = {};
    for (int i = b.lo; i < b.hi; ++i) {
        const int c = (int)sh.count[i];
        if (!c) continue;
        const double one = weight_of(k, high - i);
        if (!(one >= m) && one < 1.0) break;
        n += c;
        w += (double)c * one;
        f = {n, high - (uint32_t)i, c - 1, w, one};
    }
    // the last thread that keeps any: the tokens behind it are not kept
    const bool any = f.n > 0;
    const uint32_t last = block_max(sh, any ? (uint32_t)threadIdx.x + 1 : 0u);
    if (any && last == threadIdx.x + 1 && out->n != kAll) *out = f;
}

// One try with the window [high, low] from the row's maximum on: true and *at, *total (the drawn place, the kept
// weight) where it is certain.  rest, error: the weight below the window and its bound.
__device__ bool decide(SampleShared& sh, const Scale& k, const Wish& wish, uint32_t high, uint32_t low, bool more,
                       double rest, double error, Found* at, double* total) {
    int count;
    double sum;
    const Bins b = window_bins(sh, k, high, low, 0, 0.0, &count, &sum);
    if (threadIdx.x < 4) sh.found[threadIdx.x] = {};
    __syncthreads();
    int kept = kAll;          // tokens kept, kAll: all of the row
    double low_sum, high_sum; // bounds of the kept weight
    if (!more) rest = error = 0.0;
    // top-k
    if (wish.k <= count || !more) {
        kept = min(wish.k, count);
        find_count(sh, k, b, high, kept, &sh.found[0]);
        __syncthreads();
        low_sum = high_sum = sh.found[0].sum;
    } else if (wish.k == kAll) {
        low_sum = sum + rest - error;
        high_sum = sum + rest + error;
    } else {
        return false;  // the k-th lies below
    }
    // top-p: the place for both ends of the bound
    int kept_low = kept, kept_high = kept;
    if (wish.p < 1.0) {
        find_weight<false>(sh, k, b, high, 0, wish.p * low_sum, &sh.found[1]);
        find_weight<false>(sh, k, b, high, 0, wish.p * high_sum, &sh.found[2]);
        __syncthreads();
        const Found f1 = sh.found[1], f2 = sh.found[2];
        if (f1.n) {
            kept_low = min(kept, f1.n);
            if (f1.n <= kept) low_sum = f1.sum;
        } else if (more && kept == kAll) {
            kept_low = kBeyond;
        }
        if (f2.n) {
            kept_high = min(kept, f2.n);
            if (f2.n <= kept) high_sum = f2.sum;
        } else if (more && kept == kAll) {
            kept_high = kBeyond;
        }
        __syncthreads();
        if (threadIdx.x < 4) sh.found[threadIdx.x] = {};
        __syncthreads();
    }
    if (wish.m > 0.0) {
        find_min_p(sh, k, b, high, low, more, wish.m, &sh.found[3]);
        __syncthreads();
        const Found f = sh.found[3];
        if (f.n != kAll && f.n > 0) {
            if (f.n < kept_low) kept_low = f.n, low_sum = f.sum;
            if (f.n < kept_high) kept_high = f.n, high_sum = f.sum;
        }
    }
    if (kept_low != kept_high || kept_low == kBeyond) return false;
    if (kept_low != kAll) {
        find_count(sh, k, b, high, kept_low, &sh.found[0]);  // the last that is kept
    }
    if (wish.u < 1.0) {
        find_weight<true>(sh, k, b, high, 0, wish.u * low_sum, &sh.found[1]);
        find_weight<true>(sh, k, b, high, 0, wish.u * high_sum, &sh.found[2]);
    }
    __syncthreads();
    const Found last = sh.found[0];
    Found f1 = sh.found[1], f2 = sh.found[2];
    if (kept_low != kAll) {
        if (!f1.n || f1.n > kept_low) f1 = last;
        if (!f2.n || f2.n > kept_low) f2 = last;
    }
    if (!f1.n || f1.n != f2.n) return false;
    *at = f1;
    *total = 0.5 * (low_sum + high_sum);
    return true;
}

__device__ __forceinline__ void send(SampleShared& sh, int cluster, const Command& c) {
    // every thread of the first CTA holds the same command; the words go to all CTAs
    constexpr int kWords = sizeof(Command) / 4;
    const int tid = threadIdx.x;
    if (tid < cluster * kWords) {
        const int word = tid % kWords;
        const uint32_t v = word == 0 ? c.op : word == 1 ? c.high : word == 2 ? c.low : word == 3 ? c.rest
                         : word == 4 ? c.order : word == 5 ? c.skip : c.who;
        st_cluster(in_cta(smem_u32(&sh.cmd) + word * 4, tid / kWords), v);
    }
}

__device__ __forceinline__ void clear(SampleShared& sh, int bins) {
    for (int i = threadIdx.x; i < bins; i += kThreads) {
        sh.count[i] = 0;
        sh.lowest[i] = 0xFFFFFFFFu;
    }
}

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    SampleShared& sh = *reinterpret_cast<SampleShared*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / (unsigned)a.cluster;
    if (rank == 0) clear(sh, kBins);
    pdl_wait();
    pdl_launch_dependents();

    Slice s;
    s.row = a.logits + row * a.row_stride;
    s.vocab = a.vocab;
    s.head = min(a.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(s.row) & 15)) & 15) >> 1);
    s.pieces = (a.vocab - s.head) >> 3;
    s.tail = a.vocab - s.head - s.pieces * 8;
    s.p0 = (int)((int64_t)s.pieces * rank / a.cluster);
    s.p1 = (int)((int64_t)s.pieces * (rank + 1) / a.cluster);
    s.first = rank == 0;
    s.last = rank == (uint32_t)a.cluster - 1;

    // the row's settings
    const float temperature = a.temperature ? a.temperature[row] : 1.f;
    const bool greedy = !(temperature > 0.f);
    Wish wish;
    wish.k = a.top_k ? a.top_k[row] : 0;
    if (wish.k <= 0 || wish.k >= a.vocab) wish.k = kAll;
    if (greedy) wish.k = 1;
    const float p = a.top_p ? a.top_p[row] : 1.f, m = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    wish.p = p < 1.f ? fmax((double)p, 0.0) : 1.0;
    wish.m = m > 0.f ? (double)m : 0.0;
    wish.u = u > 0.f ? (double)u : 0.0;

    // look 1
    __half2 m2[4];
    {
        const __half2 none = as_half2(0xFC00FC00u);
#pragma unroll
        for (int i = 0; i < 4; ++i) m2[i] = none;
        each_piece(s, [&](const uint4& v, int) {
            m2[0] = max_nan2(m2[0], as_half2(v.x));
            m2[1] = max_nan2(m2[1], as_half2(v.y));
            m2[2] = max_nan2(m2[2], as_half2(v.z));
            m2[3] = max_nan2(m2[3], as_half2(v.w));
        });
        m2[0] = max_nan2(max_nan2(m2[0], m2[1]), max_nan2(m2[2], m2[3]));
    }
    const uint32_t mine = max(order16(__half_as_ushort(__low2half(m2[0]))), order16(__half_as_ushort(__high2half(m2[0]))));
    const uint32_t cta_top = block_max(sh, mine);
    // The window's reach: with a top-k the k-th largest of the threads' maxima (k logits reach it at least), else the
    // 128th, which holds the likely tokens of a trained model's row; without any limit, and for more than there are
    // threads, all of the histogram.
    const bool all = wish.k == kAll && !(wish.p < 1.0) && !(wish.m > 0.0);
    const int want = ((wish.k != kAll ? min(wish.k, kThreads * a.cluster + 1) : 128) + a.cluster - 1) / a.cluster;
    uint32_t reach = 0;
    if (greedy) {
        reach = cta_top;
    } else if (!all && want <= kThreads) {
#pragma unroll
        for (int bit = 15; bit >= 0; --bit) {
            const uint32_t t = reach | 1u << bit;
            if (__syncthreads_count(mine >= t) >= want) reach = t;
        }
    }
    if (tid < a.cluster) {
        st_cluster(in_cta(smem_u32(&sh.top[rank]), tid), cta_top);
        st_cluster(in_cta(smem_u32(&sh.reach[rank]), tid), reach);
    }
    cluster_sync();
    uint32_t top = 0, low = 0xFFFFu;
    for (int i = 0; i < a.cluster; ++i) {
        top = max(top, sh.top[i]);
        low = min(low, sh.reach[i]);
    }
    if (greedy) low = top;
    if (top >= kInfinite || top < kLowest) {  // NaN or +infinity; nothing that can be drawn
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = top >= kInfinite ? __int_as_float(0x7fffffff) : -INFINITY;
        }
        return;
    }
    Scale k;
    k.top = value_of(top);
    {
        // beyond 2^100 all but the largest logit have no weight, below 2^-100 all have the same
        const double c = fmin(fmax(1.4426950408889634074 / (greedy ? 1.0 : (double)temperature), 0x1p-100), 0x1p100);
        k.c = (float)c;
        k.c_low = (float)(c - (double)k.c);
    }
    Command cmd = {kWindow, top, max(low, window_low(top)), wish.k == kAll, 0, 0, 0};

    // first CTA: where the search is
    enum { kTry, kWide, kCollect, kTopP, kMinP, kPick };
    int stage = cmd.low == window_low(top) ? kWide : kTry;
    int windows = 0, kept = kAll, win = 0;  // win: the window that is loaded
    double kept_sum = 0.0;

    for (;;) {
        if (cmd.op == kWindow) {
            const __half low_h = __ushort_as_half((unsigned short)unorder16(cmd.low));
            const __half2 low2 = __halves2half2(low_h, low_h);
            const uint32_t counts = in_cta(smem_u32(sh.count), 0), ids = in_cta(smem_u32(sh.lowest), 0);
            __half2 b2 = as_half2(0xFC00FC00u);
            float sum = 0.f;
            each_piece(s, [&](const uint4& v, int id) {
                const uint32_t any = __hge2_mask(as_half2(v.x), low2) | __hge2_mask(as_half2(v.y), low2) |
                                     __hge2_mask(as_half2(v.z), low2) | __hge2_mask(as_half2(v.w), low2);
                if (!any) {
                    b2 = __hmax2(b2, __hmax2(__hmax2(as_half2(v.x), as_half2(v.y)), __hmax2(as_half2(v.z), as_half2(v.w))));
                    if (cmd.rest) {
                        float e[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = __half22float2(as_half2(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w));
                            e[2 * i] = ex2f((f.x - k.top) * k.c);
                            e[2 * i + 1] = ex2f((f.y - k.top) * k.c);
                        }
                        sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    }
                } else {
                    float part = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t h = half_at(v, i), o = order16(h);
                        if (o >= cmd.low) {
                            if (o <= cmd.high) {
                                add_cluster(counts + (cmd.high - o) * 4, 1u);
                                min_cluster(ids + (cmd.high - o) * 4, (uint32_t)(id + i));
                            }
                        } else {
                            const __half x = __ushort_as_half((unsigned short)h);
                            b2 = __hmax2(b2, __halves2half2(x, x));
                            if (cmd.rest) part += ex2f((__half2float(x) - k.top) * k.c);
                        }
                    }
                    sum += part;
                }
            });
            const uint32_t below = block_max(sh, max(order16(__half_as_ushort(__low2half(b2))),
                                                     order16(__half_as_ushort(__high2half(b2)))));
            double d = (double)sum;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            if (lane == 0) sh.warp_sum[warp] = d;
            __syncthreads();
            if (tid == 0) {
                d = 0.0;
                for (int i = 0; i < kWarps; ++i) d += sh.warp_sum[i];
                st_cluster(in_cta(smem_u32(&sh.rest[rank]), 0), d);
                st_cluster(in_cta(smem_u32(&sh.below[rank]), 0), below);
            }
        } else {  // tokens of one logit, warp by warp in the order of their ids
            const int n = s.p1 - s.p0, w0 = s.p0 + (int)((int64_t)n * warp / kWarps),
                      w1 = s.p0 + (int)((int64_t)n * (warp + 1) / kWarps);
            const bool edge0 = s.first && s.head && warp == 0, edge1 = s.last && s.tail && warp == kWarps - 1;
            const bool scan = cmd.op == kScan;
            if (!scan || cmd.who == rank * kWarps + warp) {
                int left = (int)cmd.skip, total = 0;
                const uint4* pc = reinterpret_cast<const uint4*>(s.row + s.head);
                // pieces -1 and w1 stand for the row's ends
                for (int base = w0 - 1; base <= w1; base += 32) {
                    const int i = base + lane;
                    int id = s.head + i * 8;
                    uint4 v = make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
                    if (i >= w0 && i < w1)
                        v = pc[i];
                    else if (i == w0 - 1 && edge0)
                        v = edge_piece(s, 0, &id);
                    else if (i == w1 && edge1)
                        v = edge_piece(s, 1, &id);
                    uint32_t hit = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) hit |= (uint32_t)(order16(half_at(v, j)) == cmd.order) << j;
                    int c = __popc(hit), run = c;
                    if (!scan) {
                        total += c;
                        continue;
                    }
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int q = __shfl_up_sync(0xffffffffu, run, d);
                        if (lane >= d) run += q;
                    }
                    const int all_hits = __shfl_sync(0xffffffffu, run, 31);
                    int skip = left - (run - c);
                    if (skip >= 0 && skip < c) {
                        for (; skip > 0; --skip) hit &= hit - 1;
                        a.token[row] = id + __ffs(hit) - 1;
                    }
                    left -= all_hits;
                    if (left < 0) break;
                }
                if (!scan) {
                    total = (int)__reduce_add_sync(0xffffffffu, (unsigned)total);
                    if (lane == 0) st_cluster(in_cta(smem_u32(&sh.ties[rank * kWarps + warp]), 0), (uint32_t)total);
                }
            }
            if (scan) return;
        }
        cluster_sync();

        if (rank == 0) {
            Command next = {kDone, 0, 0, 0, 0, 0, 0};
            if (cmd.op == kTie) {
                uint32_t at = cmd.skip, who = 0;
                while (who + 1 < (uint32_t)a.cluster * kWarps && at >= sh.ties[who]) at -= sh.ties[who++];
                next = cmd;
                next.op = kScan;
                next.skip = at;
                next.who = who;
            } else {
                uint32_t below = 0;
                double rest = 0.0;
                for (int i = 0; i < a.cluster; ++i) {
                    below = max(below, sh.below[i]);
                    rest += sh.rest[i];
                }
                const bool more = below >= kLowest;
                Found at = {};
                double total = 0.0;
                bool done = false;
                if (stage <= kWide) {
                    // A weight below the window is off by 2^-24 for each of: the sums of its thread's pieces, 3 |t|
                    // ln 2 of its exponent t (60 at most, below which all of them together are under 2^-36 of the
                    // largest's) and 4 of the power itself.
                    const double error = rest * ((double)((s.p1 - s.p0) / kThreads + 160) * 0x1p-24) +
                                         (double)a.vocab * 0x1p-60;
                    done = decide(sh, k, wish, cmd.high, cmd.low, more, rest, error, &at, &total);
                    if (!done && stage == kTry) {
                        stage = kWide;
                        next = {kWindow, top, window_low(top), wish.k == kAll, 0, 0, 0};
                    } else if (!done) {
                        stage = kCollect;
                        windows = 0;
                    }
                }
                if (!done && stage >= kCollect) {
                    // Window by window to the end, or to the k-th token: nothing is left inexact.  Then the places of
                    // top-p, min-p and the drawn token, each in the window that holds it.
                    int count;
                    double sum;
                    const int w = stage == kCollect ? windows : win;
                    const int before = w ? sh.win_count[w] : 0;
                    const double above = w ? sh.win_sum[w] : 0.0;
                    const Bins b = window_bins(sh, k, cmd.high, cmd.low, before, above, &count, &sum);
                    __syncthreads();
                    if (tid < 4) sh.found[tid] = {};
                    __syncthreads();
                    int need = -1;  // the window wanted next
                    if (stage == kCollect) {
                        if (tid == 0) {
                            sh.win_high[w] = cmd.high;
                            sh.win_low[w] = cmd.low;
                            sh.win_count[w + 1] = count;
                            sh.win_sum[w + 1] = sum;
                        }
                        windows = w + 1;
                        win = w;
                        __syncthreads();
                        if (more && count < wish.k) {
                            next = {kWindow, below, window_low(below), 0, 0, 0, 0};
                        } else {
                            kept = min(wish.k, count);
                            find_count(sh, k, b, cmd.high, kept, &sh.found[0]);
                            __syncthreads();
                            kept_sum = sh.found[0].sum;
                            stage = kTopP;
                            need = w;
                        }
                    }
                    while (next.op == kDone && !done) {
                        if (stage == kTopP) {
                            if (!(wish.p < 1.0)) {
                                stage = kMinP;
                                continue;
                            }
                            const double target = wish.p * kept_sum;
                            int v = 0;
                            while (v + 1 < windows && sh.win_sum[v + 1] < target) ++v;
                            if (v != win) {
                                need = v;
                                break;
                            }
                            __syncthreads();
                            if (tid == 0) sh.found[1] = {};
                            __syncthreads();
                            find_weight<false>(sh, k, b, cmd.high, v ? sh.win_count[v] : 0, target, &sh.found[1]);
                            __syncthreads();
                            const Found f = sh.found[1];
                            if (f.n && f.n <= kept) kept = f.n, kept_sum = f.sum;
                            stage = kMinP;
                        } else if (stage == kMinP) {
                            if (!(wish.m > 0.0)) {
                                stage = kPick;
                                continue;
                            }
                            int v = 0;
                            while (v + 1 < windows && weight_of(k, sh.win_high[v + 1]) >= wish.m) ++v;
                            if (v != win) {
                                need = v;
                                break;
                            }
                            __syncthreads();
                            if (tid == 0) sh.found[1] = {};
                            __syncthreads();
                            find_min_p(sh, k, b, cmd.high, cmd.low, false, wish.m, &sh.found[1]);
                            __syncthreads();
                            const Found f = sh.found[1];
                            if (f.n && f.n < kept) kept = f.n, kept_sum = f.sum;
                            stage = kPick;
                        } else {
                            const double target = wish.u * kept_sum;
                            int v = 0;
                            if (wish.u < 1.0)
                                while (v + 1 < windows && sh.win_sum[v + 1] <= target) ++v;
                            int v_last = 0;
                            while (v_last + 1 < windows && sh.win_count[v_last + 1] < kept) ++v_last;
                            if (!(wish.u < 1.0) || v > v_last) v = v_last;
                            if (v != win) {
                                need = v;
                                break;
                            }
                            __syncthreads();
                            if (tid < 2) sh.found[tid] = {};
                            __syncthreads();
                            if (wish.u < 1.0)
                                find_weight<true>(sh, k, b, cmd.high, v ? sh.win_count[v] : 0, target, &sh.found[1]);
                            find_count(sh, k, b, cmd.high, min(kept, count), &sh.found[0]);
                            __syncthreads();
                            at = sh.found[1];
                            if (!at.n || at.n > kept) at = sh.found[0];
                            total = kept_sum;
                            done = true;
                        }
                    }
                    if (!done && next.op == kDone) {
                        win = need;
                        next = {kWindow, sh.win_high[need], sh.win_low[need], 0, 0, 0, 0};
                    }
                }
                if (done) {
                    if (tid == 0 && a.logprob) {
                        const float2 t = power_of(k, value_of(at.order));
                        a.logprob[row] = fminf((float)(((double)t.x + (double)t.y) * 0.69314718055994530942 - log(total)), 0.f);
                    }
                    if (at.tie == 0) {
                        if (tid == 0) a.token[row] = (int64_t)sh.lowest[cmd.high - at.order];
                        next.op = kDone;
                    } else {
                        next = {kTie, 0, 0, 0, at.order, (uint32_t)at.tie, 0};
                    }
                }
            }
            __syncthreads();
            if (next.op == kWindow) clear(sh, (int)(next.high - next.low) + 1);
            send(sh, a.cluster, next);
        }
        cluster_sync();
        cmd = sh.cmd;
        if (cmd.op == kDone) return;
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs of a row: enough to fill the GPU, and of at least 4096 logits each.
int cluster_for(int64_t rows, int64_t vocab, int sms) {
    int c = 1;
    while (c < kMaxCluster && rows * c < (int64_t)sms * 2 && vocab >= (int64_t)c * 2 * 4096) c *= 2;
    return c;
}

}  // namespace

cudaError_t sample_prepare() {
    return cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SampleShared));
}

}  // namespace mnb

extern "C" int mnb_sample(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int64_t* token, float* logprob, void* stream) {
    using namespace mnb;
    if (rows < 0 || vocab < 1 || row_stride < vocab) return MNB_ERR_ARG;
    if (vocab > kMaxVocab || rows > INT32_MAX / kMaxCluster) return MNB_ERR_UNSUPPORTED;
    if (rows == 0) return MNB_OK;
    if (!logits || !u || !token) return MNB_ERR_ARG;
    if (!aligned(logits, 16) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 8) || !aligned(logprob, 4))
        return MNB_ERR_ALIGN;
    int sms;
    unsigned int* status;
    const int rc = device_ready(&sms, &status);
    if (rc != MNB_OK) return rc;
    SampleArgs a;
    a.logits = static_cast<const __half*>(logits);
    a.rows = rows;
    a.row_stride = row_stride;
    a.vocab = (int)vocab;
    a.cluster = cluster_for(rows, vocab, sms);
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.token = token;
    a.logprob = logprob;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(SampleShared);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
