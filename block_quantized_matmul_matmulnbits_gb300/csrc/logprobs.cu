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
    unsigned long long merged[kMaxCluster * kMaxTop];
    unsigned long long best[kWarpCount];
    Stat warp_stat[kWarpCount];
    Stat stat;
    int count;
};

__device__ __forceinline__ unsigned long long ld_peer_u64(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    unsigned long long v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote));
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LpArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ LpShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.cluster);
    const int64_t row = blockIdx.x / a.cluster;
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
    Stat st = {-INFINITY, 0.f, 0.f};
    uint32_t best = 0;  // order16 of this thread's largest logit
    bool ok = true;
    for (int i = 0; i < pieces; ++i) {
        ok = ok && mbar_wait(bars + 8u * i, 0, a.status);
        if (!ok) break;
        const int v = i * kThreads + tid;
        if (v >= nv) break;
        const uint4 q = *reinterpret_cast<const uint4*>(smem + (size_t)v * 16);
        const __half2 h[4] = {*reinterpret_cast<const __half2*>(&q.x), *reinterpret_cast<const __half2*>(&q.y),
                              *reinterpret_cast<const __half2*>(&q.z), *reinterpret_cast<const __half2*>(&q.w)};
        const __half2 m2 = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const __half mh = __hmax(__low2half(m2), __high2half(m2));
        best = max(best, order16(__half_as_ushort(mh)));
        const float top = __half2float(mh) * a.c;
        if (top > st.r + kMove || st.r == -INFINITY) {
            if (top != -INFINITY && top == top) {
                const Stat none = {top, 0.f, 0.f};
                st = join(st, none);
            }
        }
        const float r = st.r == -INFINITY ? 0.f : st.r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            const float y0 = max_nan(fmaf(f.x, a.c, -r), -200.f), y1 = max_nan(fmaf(f.y, a.c, -r), -200.f);
            const float e0 = ex2f(y0), e1 = ex2f(y1);
            st.z += e0 + e1;
            st.y = fmaf(e0, y0, st.y);
            st.y = fmaf(e1, y1, st.y);
        }
    }
    // every copy has landed before anything below may end the CTA
    for (int i = 0; i < pieces; ++i)
        if (!mbar_wait(bars + 8u * i, 0, a.status, false)) break;

    Stat ws = st;
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
        sh.stat = s;
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
                const uint4 q = *reinterpret_cast<const uint4*>(smem + (size_t)v * 16);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t o = order16((w[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu);
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

    // ---- the cluster's first CTA joins
    __syncthreads();
    if (a.cluster > 1) cluster_sync();
    if (rank == 0) {
        const uint32_t s_top = smem_u32(sh.top), s_stat = smem_u32(&sh.stat);
        const int nk = a.cluster * a.top;
        for (int i = tid; i < nk; i += kThreads) sh.merged[i] = ld_peer_u64(s_top + 8u * (i % a.top), (uint32_t)(i / a.top));
        Stat s = sh.stat;
        for (int q = 1; q < a.cluster; ++q) {
            Stat o;
            o.r = ld_peer_f32(s_stat, (uint32_t)q);
            o.z = ld_peer_f32(s_stat + 4u, (uint32_t)q);
            o.y = ld_peer_f32(s_stat + 8u, (uint32_t)q);
            s = join(s, o);
        }
        __syncthreads();
        const bool none = s.z == 0.f && s.r == -INFINITY;
        const float logz = log2f(s.z);
        const float bad = s.z != s.z || s.z == INFINITY ? __int_as_float(0x7fffffff) : 0.f;
        auto logp = [&](float x) { return none ? -INFINITY : (fmaf(x, a.c, -s.r) - logz) * kLn2f + bad; };
        for (int i = tid; i < nk; i += kThreads) {
            const unsigned long long k = sh.merged[i];
            int above = 0;
            for (int j = 0; j < nk; ++j) above += sh.merged[j] > k;
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
    if (a.cluster > 1) cluster_sync();  // the peers' lists stay until they are read
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
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel, a) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
