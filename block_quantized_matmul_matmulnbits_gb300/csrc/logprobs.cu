// logprobs.cu -- log probability of a given token, entropy and the most likely
// tokens of each row of logits (mnb_logprobs).
//
// One thread-block cluster takes a row, each of its CTAs a slice, each thread
// every 256th 16-byte piece of it, straight from memory into registers, in groups of
// three pieces of which the next is on its way (32.7 us in the case below when this was chosen, four a
// group 34.3, two 35.2).  Every thread keeps sum 2^y and sum 2^y y of y = x c - r,
// c = scale log2(e), with a reference r of its own: the largest value seen, which moves only when
// a value passes it by 5.75 (moving at once, 33.5 us; by 8, 32.7).  Any r near the row's maximum serves the sums, but the entropy is a
// difference of two terms, each as far from it as r from the maximum: with the maximum itself, which a
// row with one likely token has for r, it loses nothing (with one 4 above
// the maximum four times the error, over 40 such rows).  The threads' sums are brought to a
// common reference at the end:
//     lse = ln 2 (M + log2 Z),   entropy = ln 2 (log2 Z - (sum 2^y y) / Z).
// A thread's fixed work (joining, selecting) costs as much as about 100 logits,
// so a row gets no more CTAs than the GPU needs to be full.
//
// The k most likely: the k-th largest of the threads' own maxima is a value
// that at least k of the CTA's logits reach.  Each thread remembers which two
// groups of pieces held its largest logits and the largest of the others, so few groups
// have to be looked at again, a piece a thread, and all of a thread's only where a third
// one reaches that value too; what reaches it is collected, and ranks among
// the collected are counted directly.  FP16 logits tie often; the keys order
// equal ones by rising id.  Where more are collected than the list holds (long
// runs of equal logits), the CTA takes its maximum k times instead.  The cluster's
// first CTA merges the lists that the others leave in its shared memory.
//
// Bound by memory: 2 bytes a logit, read once.  512 rows of 151,936 with the 20 most likely:
// 33.1 us, 4.7 TB/s; without them 29.5 us, 5.3 TB/s.  All rows end at about the same time,
// so what follows the last logit (the k-th largest bit by bit, the second look, the
// ranks) is not hidden by another row's loads; more CTAs a row, that would hide it,
// cost more than that in fixed work (two a row: 41 us).
//
// With a scale so large that a place of FP32 at 65504 c is worth more than a unit, r = x c is no
// longer the largest logit's (from 2^31 on that one's term could be 2^64 and more).  There the
// reference is the logit itself and y = (x - r) c:
// two roundings a logit instead of one, and no distance kept (35.8 us in the case above; the
// first form with the largest scale it takes 33.0).
#include <cuda_fp16.h>

#include "common.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpCount = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 512;              // candidates of a CTA
constexpr int kMaxVocab = 1 << 24;
constexpr int kUnroll = 3;              // pieces of a group; two groups in registers
constexpr float kMove = 5.75f;          // 4 in natural units
constexpr float kMostScale = 256.f;     // c of the first form: a place of FP32 below 65504 * 256 is a unit

constexpr float kLn2f = 0.693147180559945309417f;

struct LpArgs {
    const __half* logits;
    int64_t rows, row_stride;
    int vocab, top, cluster;
    float c;  // scale * log2(e)
    const int64_t* target;
    float *logprob, *entropy, *top_logprobs;
    int32_t* top_ids;
};

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// FP16 bits as an unsigned value in the same order (-0 counts as +0, a NaN of any kind as the
// largest); never 0.
__device__ __forceinline__ uint32_t order16(uint32_t h) {
    h = h == 0x8000u ? 0u : h;
    h = (h & 0x7FFFu) > 0x7C00u ? 0x7FFFu : h;
    return (h & 0x8000u) ? (~h & 0xFFFFu) : (h | 0x8000u);
}

__device__ __forceinline__ uint32_t unorder16(uint32_t o) { return (o & 0x8000u) ? (o & 0x7FFFu) : (~o & 0xFFFFu); }

// Larger logit first, then the lower id; 0 is no candidate.
__device__ __forceinline__ unsigned long long key_of(uint32_t order, uint32_t id) {
    return ((unsigned long long)order << 32) | (uint32_t)~id;
}

struct Stat {  // sums about the reference r (times `unit`: in units of log2)
    float r, z, y;
};

// The same sums about another reference, not below r.  One of -infinity comes with sums of
// 0 (or NaN) and has no shift of its own.
__device__ __forceinline__ Stat about(const Stat& s, float r, float unit) {
    const float d = fmaxf((s.r - (r == -INFINITY ? 0.f : r)) * unit, -1000.f), f = ex2f(d);
    return {r, s.z * f, f * fmaf(s.z, d, s.y)};
}

__device__ __forceinline__ Stat warp_join(Stat s, float unit) {
    float r = s.r;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, x));
    s = about(s, r, unit);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        s.z += __shfl_xor_sync(0xffffffffu, s.z, x);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, x);
    }
    return s;
}

struct __align__(16) LpShared {
    unsigned long long list[kList];
    unsigned long long top[kMaxTop];       // this CTA's best, sorted
    unsigned long long merged[kMaxCluster * kMaxTop];  // first CTA: every CTA's best, sorted each
    unsigned long long best[kWarpCount];
    Stat warp_stat[kWarpCount];
    Stat stats[kMaxCluster];               // first CTA: every CTA's sums
    int work[2 * kThreads];                // first pieces of groups to look at again
    int count, works;
};

// The address that `addr` of this CTA has in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Pairs of binary32 values in one 64-bit register: one instruction for two.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

__device__ __forceinline__ __half2 max_of(const uint4& q) {
    return __hmax2(__hmax2(as_half2(q.x), as_half2(q.y)), __hmax2(as_half2(q.z), as_half2(q.w)));
}

__device__ __forceinline__ uint32_t order_of(float x) { return order16(__half_as_ushort(__float2half_rn(x))); }

__device__ __forceinline__ uint4 ld_stream(const void* p) {  // once, from memory
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// The running sums and the largest logits of one thread, a group of up to kUnroll pieces
// at a time.  FINE: the reference is a logit and c its unit; else it is in units of log2.
template <bool FINE>
struct Look {
    float r = -INFINITY;                // reference
    uint64_t z2 = 0, y2 = 0, ref2 = 0;  // both sums in two halves; (-r, -r), 0 while r is -infinity
    float best = -INFINITY, second = -INFINITY, third = -INFINITY;  // the three largest of the groups' maxima
    int at = -1, second_at = -1;        // first pieces of the first two's groups

    template <int N>
    __device__ __forceinline__ void add(const uint4 (&q)[N], int v, float c, uint64_t c2) {
        __half2 m2 = max_of(q[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) m2 = __hmax2(m2, max_of(q[i]));
        const float x = __half2float(__hmax(__low2half(m2), __high2half(m2)));
        third = fmaxf(third, fminf(second, x));
        second_at = x > best ? at : (x > second ? v : second_at);
        second = fmaxf(second, fminf(best, x));
        at = x > best ? v : at;
        best = fmaxf(best, x);
        const float top = FINE ? x : x * c;
        if (top > (FINE ? r : r + kMove)) {  // never for a NaN
            const float to = top;
            const float d = fmaxf(FINE ? (r - to) * c : r - to, -1000.f), f = ex2f(d);
            const float2 zz = unpair(z2), yy = unpair(y2);
            z2 = pair(zz.x * f, zz.y * f);
            y2 = pair(f * fmaf(zz.x, d, yy.x), f * fmaf(zz.y, d, yy.y));
            r = to;
            ref2 = pair(-to, -to);
        }
        // 0 times -infinity has to stay 0.  Where FP16's lowest value adds nothing (2^-160 of
        // the reference), -infinity is replaced by it, two logits at a time; else the
        // exponents are held at -200 one by one.
        if (!FINE && r >= fmaf(-65504.f, c, 160.f))
            sum<false>(q, c2);
        else
            sum<true>(q, c2);
    }

    template <bool LOW, int N>
    __device__ __forceinline__ void sum(const uint4 (&q)[N], uint64_t c2) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 h = LOW ? as_half2(w[j]) : __hmax2_nan(as_half2(w[j]), as_half2(0xFBFFFBFFu));
                const float2 f = __half22float2(h);
                float2 y = unpair(FINE ? mul2(add2(pair(f.x, f.y), ref2), c2) : fma2(pair(f.x, f.y), c2, ref2));
                if (LOW) y = make_float2(max_nan(y.x, -200.f), max_nan(y.y, -200.f));
                const uint64_t e = pair(ex2f(y.x), ex2f(y.y));
                z2 = add2(z2, e);
                y2 = fma2(e, pair(y.x, y.y), y2);
            }
        }
    }
};

template <bool FINE>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LpArgs a) {
    __shared__ LpShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.cluster);
    const int64_t row = blockIdx.x / a.cluster;
    if (a.cluster > 1) cluster_arrive();  // waited for before the first CTA's memory is written
    if (tid == 0) sh.count = sh.works = 0;
    pdl_wait();
    pdl_launch_dependents();
    const __half* src = a.logits + row * a.row_stride;
    // The row in 16-byte pieces from the boundary at or before its start: element e of
    // piece v is token 8 v + e - skew.  Pieces f0 .. f1 - 1 of this CTA's v0 .. v1 - 1 lie wholly
    // in the row; at most one at either end of the row is ragged.
    const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15u) >> 1);
    const int vecs = (a.vocab + skew + 7) >> 3;
    const int v0 = (int)((int64_t)rank * vecs / a.cluster), v1 = (int)((int64_t)(rank + 1) * vecs / a.cluster);
    const int f0 = max(v0, skew > 0 ? 1 : 0), f1 = min(v1, (a.vocab + skew) >> 3);
    const __half* pieces = src - skew;
    auto token = [&](int v, int e) { return (int64_t)v * 8 + e - skew; };
    auto logit = [&](int64_t id) {  // -infinity outside the row
        return id >= 0 && id < a.vocab ? (uint32_t)__half_as_ushort(src[id]) : 0xFC00u;
    };
    auto piece = [&](int v) {
        if (v >= f0 && v < f1) return ld_stream(pieces + (int64_t)v * 8);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = logit(token(v, 2 * j)) | (logit(token(v, 2 * j + 1)) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // the keys of a piece's tokens that are in the row and reach `least`
    auto each = [&](const uint4& x, int v, uint32_t least, auto&& take) {
        const __half2 m2 = max_of(x);
        if (order16(__half_as_ushort(__hmax(__low2half(m2), __high2half(m2)))) < least) return;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t id = token(v, e);
            const uint32_t o = order16((w[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu);
            if (o >= least && id >= 0 && id < a.vocab) take(key_of(o, (uint32_t)id));
        }
    };

    // ---- one look at the slice
    Look<FINE> look;
    const float unit = FINE ? a.c : 1.f;
    const uint64_t c2 = pair(a.c, a.c);
    bool any = f0 + tid < f1;  // this thread has a piece
    // the ragged pieces: the slice's first belongs to thread 0 too, its last to thread 1
    const int edge = tid == 0 ? v0 : v1 - 1;
    const bool ragged = tid < 2 && v1 > v0 && (edge < f0 || edge >= f1) && (tid == 0 || v1 - 1 > v0);
    if (ragged) {
        const uint4 one[1] = {piece(edge)};
        look.add(one, edge, a.c, c2);
        any = true;
    }
    int v = f0 + tid;
    constexpr int kStep = kUnroll * kThreads;
    uint4 q[2][kUnroll];  // a group, and the next one on its way
    auto fetch = [&](uint4(&to)[kUnroll], int v) {
        if (v + (kUnroll - 1) * kThreads < f1) {
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) to[j] = ld_stream(pieces + (int64_t)(v + j * kThreads) * 8);
        }
    };
    fetch(q[0], v);
    while (v + (kUnroll - 1) * kThreads < f1) {
        fetch(q[1], v + kStep);
        look.add(q[0], v, a.c, c2);
        v += kStep;
        if (v + (kUnroll - 1) * kThreads >= f1) break;
        fetch(q[0], v + kStep);
        look.add(q[1], v, a.c, c2);
        v += kStep;
    }
    {  // fewer than a group are left: all on their way before the first is looked at
        uint4 rest[kUnroll - 1];
#pragma unroll
        for (int j = 0; j < kUnroll - 1; ++j)
            if (v + j * kThreads < f1) rest[j] = ld_stream(pieces + (int64_t)(v + j * kThreads) * 8);
#pragma unroll
        for (int j = 0; j < kUnroll - 1; ++j)
            if (v + j * kThreads < f1) {
                const uint4 one[1] = {rest[j]};
                look.add(one, v + j * kThreads, a.c, c2);
            }
    }

    const float2 zs = unpair(look.z2), ys = unpair(look.y2);
    Stat ws = {look.r, zs.x + zs.y, ys.x + ys.y};
    ws = warp_join(ws, unit);
    if (lane == 0) sh.warp_stat[warp] = ws;
    if (tid < kMaxTop) sh.top[tid] = 0;
    __syncthreads();
    if (warp == 0) {
        Stat s = {-INFINITY, 0.f, 0.f};
        if (lane < kWarpCount) s = sh.warp_stat[lane];
        s = warp_join(s, unit);
        if (lane == 0) sh.stats[0] = s;
    }

    // ---- this CTA's k best
    if (a.top > 0) {
        uint32_t tau = 0;  // the k-th largest of the threads' maxima, bit by bit
        const uint32_t best = any ? order_of(look.best) : 0u;
#pragma unroll
        for (int bit = 15; bit >= 0; --bit) {
            const uint32_t t = tau | (1u << bit);
            if (__syncthreads_count(best >= t) >= a.top) tau = t;
        }
        auto collect = [&](const uint4& x, int v) {
            each(x, v, tau, [&](unsigned long long k) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.list[at] = k;
            });
        };
        const bool reach = any && best >= tau;
        const bool two = order_of(look.second) >= tau;
        const bool all = reach && (look.at < 0 || order_of(look.third) >= tau || (two && look.second_at < 0));
        if (reach && !all) {
            const int i = atomicAdd(&sh.works, two ? 2 : 1);
            sh.work[i] = look.at;
            if (two) sh.work[i + 1] = look.second_at;
        }
        __syncthreads();
        // a piece a thread; an entry is a whole group, or the single piece at an end of the slice
        for (int i = tid; i < sh.works * kUnroll; i += kThreads) {
            const int from = sh.work[i / kUnroll], v = from + i % kUnroll * kThreads;
            if (v == from || (from >= f0 && from + (kUnroll - 1) * kThreads < f1)) collect(piece(v), v);
        }
        if (all && ragged) collect(piece(edge), edge);
        // a thread's whole pieces are looked at by its warp, two a lane at a time
        for (unsigned left = __ballot_sync(0xffffffffu, all); left; left &= left - 1) {
            int v = f0 + warp * 32 + (__ffs(left) - 1) + lane * kThreads;
            for (; v < f1; v += 64 * kThreads) {
                const int w = v + 32 * kThreads;
                const uint4 x = ld_stream(pieces + (int64_t)v * 8);
                const uint4 y = w < f1 ? ld_stream(pieces + (int64_t)w * 8) : x;
                collect(x, v);
                if (w < f1) collect(y, w);
            }
        }
        __syncthreads();
        const int n = sh.count;
        if (n <= kList) {  // the order of the list does not matter: the keys differ
            for (int i = tid; i < n; i += kThreads) {
                const unsigned long long k = sh.list[i];
                int above = 0;
                for (int j = 0; j < n; ++j) above += sh.list[j] > k;
                if (above < a.top) sh.top[above] = k;
            }
        } else {
            unsigned long long last = ~0ull;
            for (int j = 0; j < a.top; ++j) {
                unsigned long long mine = 0;
                for (int v = v0 + tid; v < v1; v += kThreads)
                    each(piece(v), v, 0u, [&](unsigned long long k) { mine = k < last && k > mine ? k : mine; });
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) {
                    const unsigned long long o = __shfl_xor_sync(0xffffffffu, mine, x);
                    mine = o > mine ? o : mine;
                }
                __syncthreads();
                if (lane == 0) sh.best[warp] = mine;
                __syncthreads();
                last = 0;
                for (int w = 0; w < kWarpCount; ++w) last = sh.best[w] > last ? sh.best[w] : last;
                if (tid == 0) sh.top[j] = last;
                if (last == 0) break;  // the whole CTA together
            }
        }
    }

    // ---- the cluster's first CTA joins what the others leave in its memory
    __syncthreads();
    if (a.cluster > 1) {
        cluster_wait();
        if (rank > 0) {
            const uint32_t dst = in_first(smem_u32(sh.merged)) + 8u * (uint32_t)(rank * a.top);
            for (int i = tid; i < a.top; i += kThreads)
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst + 8u * i), "l"(sh.top[i]) : "memory");
            if (tid == 0) {
                const uint32_t to = in_first(smem_u32(&sh.stats[rank]));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(sh.stats[0].r) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4u), "f"(sh.stats[0].z) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8u), "f"(sh.stats[0].y) : "memory");
            }
        } else {
            for (int i = tid; i < a.top; i += kThreads) sh.merged[i] = sh.top[i];
        }
        cluster_arrive();
        if (rank > 0) return;
        cluster_wait();
    } else {
        for (int i = tid; i < a.top; i += kThreads) sh.merged[i] = sh.top[i];
        __syncthreads();
    }
    {
        const int nk = a.cluster * a.top;
        Stat s = {-INFINITY, 0.f, 0.f};
        if (lane < a.cluster) s = sh.stats[lane];
        s = warp_join(s, unit);
        const bool none = s.z == 0.f && s.r == -INFINITY;
        const float logz = log2f(s.z);
        const float bad = s.z != s.z || s.z == INFINITY ? __int_as_float(0x7fffffff) : 0.f;
        auto logp = [&](float x) {
            const float y = FINE ? (x - s.r) * a.c : fmaf(x, a.c, -s.r);
            return none ? -INFINITY : (y - logz) * kLn2f + bad;
        };
        for (int i = tid; i < nk; i += kThreads) {
            // every list is sorted: its keys above k are found by halving, all lists at once
            const unsigned long long k = sh.merged[i];
            int above = 0;
#pragma unroll
            for (int q = 0; q < kMaxCluster; ++q) {
                if (q >= a.cluster) break;
                int lo = 0, hi = a.top;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sh.merged[q * a.top + mid] > k)
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                above += lo;
            }
            if (k != 0 && above < a.top) {
                a.top_ids[row * a.top + above] = (int32_t)~(uint32_t)k;
                a.top_logprobs[row * a.top + above] =
                    logp(__half2float(__ushort_as_half((unsigned short)unorder16((uint32_t)(k >> 32)))));
            }
        }
        if (tid == 0) {
            if (a.entropy) a.entropy[row] = none ? 0.f : (logz - __fdiv_rn(s.y, s.z)) * kLn2f + bad;
            if (a.target) {
                const int64_t id = a.target[row];
                a.logprob[row] = id >= 0 && id < a.vocab ? logp(__half2float(src[id])) : 0.f;
            }
        }
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs of a row: enough for two on every SM (four fit), of at least 2048 logits each.  With more
// their fixed work costs more than fuller SMs give (200 rows of 151,936: 20.9 us with two a
// row, 25.4 with four; 300 rows: 22.4 with one, 33.8 with two).
int cluster_for(int64_t rows, int64_t vocab, int sms) {
    int c = 1;
    while (c < kMaxCluster && rows * c < (int64_t)sms * 2 && vocab >= (int64_t)c * 2 * 2048) c *= 2;
    return c;
}

}  // namespace

}  // namespace mnb

extern "C" int mnb_logprobs(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride, float scale,
                            const int64_t* target, int32_t top, float* logprob, float* entropy, int32_t* top_ids,
                            float* top_logprobs, void* stream) {
    using namespace mnb;
    if (rows < 0 || vocab < 1 || row_stride < vocab || top < 0 || top > vocab || !(scale > 0.f) || scale > 2e38f)
        return MNB_ERR_ARG;
    if (vocab > kMaxVocab || top > kMaxTop || rows > INT32_MAX / kMaxCluster) return MNB_ERR_UNSUPPORTED;
    if (rows == 0) return MNB_OK;
    if (!logits || (target && !logprob) || (top > 0 && (!top_ids || !top_logprobs))) return MNB_ERR_ARG;
    if (!aligned(logits, 16) || !aligned(target, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return MNB_ERR_ALIGN;
    int sms;
    unsigned int* status;
    const int rc = device_ready(&sms, &status);
    if (rc != MNB_OK) return rc;
    LpArgs a;
    a.logits = static_cast<const __half*>(logits);
    a.rows = rows;
    a.row_stride = row_stride;
    a.vocab = (int)vocab;
    a.top = top;
    a.cluster = cluster_for(rows, vocab, sms);
    a.c = scale * 1.44269504088896340736f;
    a.target = target;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
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
    const auto kernel = a.c > kMostScale ? logprobs_kernel<true> : logprobs_kernel<false>;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
