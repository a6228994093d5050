// logprobs.cu -- log probability of a given token, entropy and the most likely
// tokens of each row of logits (mnb_logprobs).
//
// One thread-block cluster takes a row; each CTA copies a slice of it into
// shared memory (bulk copies of 4 KB, one barrier each) and reads it as the
// pieces arrive.  Every thread keeps sum 2^(x c - r) and sum 2^(x c - r) (x c - r),
// c = scale log2(e), with a reference r of its own: any r near the row's
// maximum serves, so it is moved only when a value passes it by 2^4 (what the
// entropy's difference of two terms can lose to it stays at 4 roundings of 1),
// and the threads' sums are brought to a common one at the end:
//     lse = ln 2 (M + log2 Z),   entropy = ln 2 (log2 Z - (sum 2^y y) / Z),   y = x c - M.
//
// The k most likely: the k-th largest of the threads' own maxima is a value
// that at least k of the CTA's logits reach, so only the few threads whose
// maximum reaches it look at their logits again (in shared memory) and collect
// those that do; ranks among the collected are counted directly.  FP16
// logits tie often; the keys order equal ones by rising id.  Where more are collected
// than the list holds (long runs of equal logits), the CTA takes its maximum k
// times instead.  The cluster's first CTA merges the CTAs' lists through
// distributed shared memory.
//
// Bound by memory: 2 bytes a logit, read once.  A slice is at most 40 KB where
// eight CTAs a cluster allow it, so that several CTAs share an SM and one's
// selection runs under the others' copies.
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
constexpr int64_t kMaxVocab = 786432;   // eight slices of 192 KB
constexpr uint32_t kSliceTarget = 40960;
constexpr float kMove = 4.f;
constexpr float kLn2f = 0.693147180559945309417f;

struct LpArgs {
    const __half* logits;
    int64_t rows, row_stride;
    int vocab, top, cluster;
    int slice_vecs;  // 16-byte pieces of shared memory a CTA
    float c;         // scale * log2(e)
    const int64_t* target;
    float *logprob, *entropy, *top_logprobs;
    int32_t* top_ids;
    unsigned int* status;
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

struct Stat {  // sums about the reference r (in units of log2)
    float r, z, y;
};

__device__ __forceinline__ Stat join(Stat a, Stat b) {
    Stat s;
    s.r = fmaxf(a.r, b.r);
    const float u = s.r == -INFINITY ? 0.f : s.r;
    // a reference of -infinity comes with sums of 0 (or NaN): no shift of its own
    const float da = fmaxf(a.r - u, -1000.f), db = fmaxf(b.r - u, -1000.f);
    const float fa = ex2f(da), fb = ex2f(db);
    s.z = a.z * fa + b.z * fb;
    s.y = fa * (a.y + a.z * da) + fb * (b.y + b.z * db);
    return s;
}

struct __align__(16) LpShared {
    unsigned long long bars[64];           // one a 4 KB piece
    unsigned long long list[kList];
    unsigned long long top[kMaxTop];       // this CTA's best, sorted
    unsigned long long merged[kMaxCluster * kMaxTop];  // first CTA: every CTA's best, sorted each
    unsigned long long best[kWarpCount];
    Stat warp_stat[kWarpCount];
    Stat stats[kMaxCluster];               // first CTA: every CTA's sums
    int count;
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

__device__ __forceinline__ uint32_t max_order(const uint4& q) {  // order16 of a piece's largest logit
    const __half2 m2 = __hmax2(__hmax2(*reinterpret_cast<const __half2*>(&q.x), *reinterpret_cast<const __half2*>(&q.y)),
                               __hmax2(*reinterpret_cast<const __half2*>(&q.z), *reinterpret_cast<const __half2*>(&q.w)));
    return order16(__half_as_ushort(__hmax(__low2half(m2), __high2half(m2))));
}

__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LpArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ LpShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.cluster);
    const int64_t row = blockIdx.x / a.cluster;
    if (a.cluster > 1) cluster_arrive();  // waited for before the first CTA's memory is written
    pdl_wait();
    pdl_launch_dependents();
    const __half* src = a.logits + row * a.row_stride;
    // The row in 16-byte pieces from the boundary at or before its start: element e of
    // piece v is token 8 v + e - skew.  Pieces that lie wholly in the row are copied in
    // bulk, the ragged ones at its ends element by element.
    const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15u) >> 1);
    const int vecs = (a.vocab + skew + 7) >> 3;
    const int v0 = (int)((int64_t)rank * vecs / a.cluster), v1 = (int)((int64_t)(rank + 1) * vecs / a.cluster);
    const int nv = v1 - v0;
    const int f0 = max(v0, skew > 0 ? 1 : 0), f1 = min(v1, (a.vocab + skew) >> 3);  // whole pieces
    const int pieces = (nv + kThreads - 1) / kThreads;
    const uint32_t sbase = smem_u32(smem), bars = smem_u32(sh.bars);
    if (tid == 0) {
        for (int i = 0; i < pieces; ++i) mbar_init(bars + 8u * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.count = 0;
        for (int i = 0; i < pieces; ++i) {
            const int p0 = max(v0 + i * kThreads, f0), p1 = min(v0 + (i + 1) * kThreads, f1);
            if (p1 > p0) {
                mbar_arrive_tx(bars + 8u * i, (uint32_t)(p1 - p0) * 16u);
                bulk_load(sbase + (uint32_t)(p0 - v0) * 16u, src + ((int64_t)p0 * 8 - skew), (uint32_t)(p1 - p0) * 16u,
                          bars + 8u * i);
            } else {
                mbar_arrive(bars + 8u * i);
            }
        }
    }
    // the ragged pieces: at most the row's first and last, with -infinity around the row
    if (warp == 1 && lane < 16) {
        const int v = lane < 8 ? v0 : v1 - 1, e = lane & 7;
        if (nv > 0 && (v < f0 || v >= f1) && (lane < 8 || v1 - 1 > v0)) {
            const int64_t id = (int64_t)v * 8 + e - skew;
            const __half x = id >= 0 && id < a.vocab ? src[id] : __ushort_as_half((unsigned short)0xFC00u);
            reinterpret_cast<__half*>(smem)[(v - v0) * 8 + e] = x;
        }
    }
    __syncthreads();

    // ---- one look at the slice
    float r = -INFINITY;                       // the reference
    uint64_t z2 = 0, y2 = 0, ref2 = 0;         // both sums in two halves; -r, 0 while r is -infinity
    const uint64_t c2 = pair(a.c, a.c);
    uint32_t best = 0;  // order16 of this thread's largest logit
    bool ok = true;
    for (int i = 0; i < pieces; ++i) {
        ok = ok && mbar_wait(bars + 8u * i, 0, a.status);
        if (!ok) break;
        const int v = i * kThreads + tid;
        if (v >= nv) break;
        const uint4 q = *reinterpret_cast<const uint4*>(smem + (size_t)v * 16);
        const uint32_t order = max_order(q);
        best = max(best, order);
        const float top = __half2float(__ushort_as_half((unsigned short)unorder16(order))) * a.c;
        if (top > r + kMove) {  // never for a NaN
            const float f = ex2f(fmaxf(r - top, -1000.f));
            const float2 zz = unpair(z2), yy = unpair(y2);
            const float d = fmaxf(r - top, -1000.f);
            z2 = pair(zz.x * f, zz.y * f);
            y2 = pair(f * fmaf(zz.x, d, yy.x), f * fmaf(zz.y, d, yy.y));
            r = top;
            ref2 = pair(-top, -top);
        }
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            const float2 y = unpair(fma2(pair(f.x, f.y), c2, ref2));
            const float y0 = max_nan(y.x, -200.f), y1 = max_nan(y.y, -200.f);
            const uint64_t e = pair(ex2f(y0), ex2f(y1));
            z2 = add2(z2, e);
            y2 = fma2(e, pair(y0, y1), y2);
        }
    }
    // every copy has landed before anything below may end the CTA
    for (int i = 0; i < pieces; ++i)
        if (!mbar_wait(bars + 8u * i, 0, a.status, false)) break;

    const float2 zs = unpair(z2), ys = unpair(y2);
    Stat ws = {r, zs.x + zs.y, ys.x + ys.y};
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        Stat o;
        o.r = __shfl_xor_sync(0xffffffffu, ws.r, x);
        o.z = __shfl_xor_sync(0xffffffffu, ws.z, x);
        o.y = __shfl_xor_sync(0xffffffffu, ws.y, x);
        ws = join(ws, o);
    }
    if (lane == 0) sh.warp_stat[warp] = ws;
    if (tid < kMaxTop) sh.top[tid] = 0;
    __syncthreads();
    if (tid == 0) {
        Stat s = sh.warp_stat[0];
        for (int w = 1; w < kWarpCount; ++w) s = join(s, sh.warp_stat[w]);
        sh.stats[0] = s;
    }

    // ---- this CTA's k best
    if (a.top > 0) {
        uint32_t tau = 0;  // the k-th largest of the threads' maxima, bit by bit
#pragma unroll
        for (int bit = 15; bit >= 0; --bit) {
            const uint32_t t = tau | (1u << bit);
            if (__syncthreads_count(best >= t) >= a.top) tau = t;
        }
        if (best >= tau && best > 0) {
            for (int v = tid; v < nv; v += kThreads) {
                if (max_order(*reinterpret_cast<const uint4*>(smem + (size_t)v * 16)) < tau) continue;
                for (int e = 0; e < 8; ++e) {
                    const uint32_t o = order16(reinterpret_cast<const unsigned short*>(smem)[v * 8 + e]);
                    const int64_t id = (int64_t)(v0 + v) * 8 + e - skew;
                    if (o >= tau && id >= 0 && id < a.vocab) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kList) sh.list[at] = key_of(o, (uint32_t)id);
                    }
                }
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
                for (int v = tid; v < nv; v += kThreads) {
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t o = order16(reinterpret_cast<const unsigned short*>(smem)[v * 8 + e]);
                        const int64_t id = (int64_t)(v0 + v) * 8 + e - skew;
                        const unsigned long long k = key_of(o, (uint32_t)id);
                        if (id >= 0 && id < a.vocab && k < last && k > mine) mine = k;
                    }
                }
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
        Stat s = sh.stats[0];
        for (int q = 1; q < a.cluster; ++q) s = join(s, sh.stats[q]);
        const bool none = s.z == 0.f && s.r == -INFINITY;
        const float logz = log2f(s.z);
        const float bad = s.z != s.z || s.z == INFINITY ? __int_as_float(0x7fffffff) : 0.f;
        auto logp = [&](float x) { return none ? -INFINITY : (fmaf(x, a.c, -s.r) - logz) * kLn2f + bad; };
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

// CTAs of a row: enough for slices of at most 40 KB, and while the rows leave
// SMs idle as many as eight with 1 KB each.
int cluster_for(int64_t rows, int64_t vocab, int sms) {
    int c = 1;
    while (c < kMaxCluster && vocab * 2 > (int64_t)c * kSliceTarget) c *= 2;
    while (c < kMaxCluster && rows * c * 2 <= sms && vocab * 2 >= (int64_t)c * 2 * 1024) c *= 2;
    return c;
}

}  // namespace

cudaError_t logprobs_prepare() {
    return cudaFuncSetAttribute(logprobs_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(kMaxVocab / kMaxCluster * 2 + 64));
}

}  // namespace mnb

extern "C" int mnb_logprobs(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride, float scale,
                            const int64_t* target, int32_t top, float* logprob, float* entropy, int32_t* top_ids,
                            float* top_logprobs, void* stream) {
    using namespace mnb;
    if (rows < 0 || vocab < 1 || row_stride < vocab || top < 0 || top > vocab || !(scale > 0.f) || scale > 3e38f)
        return MNB_ERR_ARG;
    if (vocab > kMaxVocab || top > kMaxTop || rows > INT32_MAX / kMaxCluster) return MNB_ERR_UNSUPPORTED;
    if (rows == 0) return MNB_OK;
    if (!logits || (target && !logprob) || (top > 0 && (!top_ids || !top_logprobs))) return MNB_ERR_ARG;
    if (!aligned(logits, 16) || !aligned(target, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return MNB_ERR_ALIGN;
    int sms;
    LpArgs a;
    const int rc = device_ready(&sms, &a.status);
    if (rc != MNB_OK) return rc;
    a.logits = static_cast<const __half*>(logits);
    a.rows = rows;
    a.row_stride = row_stride;
    a.vocab = (int)vocab;
    a.top = top;
    a.cluster = cluster_for(rows, vocab, sms);
    a.slice_vecs = (int)(((vocab + 7 + 7) / 8 + a.cluster - 1) / a.cluster);
    a.c = scale * 1.44269504088896340736f;
    a.target = target;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)a.slice_vecs * 16;
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel, a) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
