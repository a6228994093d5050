// kv_batch.cuh -- the paged 8-bit cache and the batch of sequences as the
// kernels see them, and how a kernel finds the sequence of its work item.
// The kernels start before the work ahead of them on the stream has finished
// and wait for it (pdl_wait); what that work may have written is read with plain
// loads, which the compiler keeps behind the wait, never with __ldg.
#pragma once

#include <stdint.h>

#include "mnb_internal.h"

namespace mnb {

// Launch that may start before the preceding kernel on the stream has finished; the
// kernel waits for it (pdl_wait) before it reads or writes anything.
template <typename A>
inline cudaError_t launch_pdl(void (*kernel)(A), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A& args,
                              int cluster_z = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 1;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = (unsigned)cluster_z;
    cfg.attrs = at;
    cfg.numAttrs = cluster_z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

constexpr int kKvBlock = MNB_KV_BLOCK;  // tokens that share a scale

// Positions of a sequence that are ever visited: a kernel's tiles and stages reach past the last
// one by less than 4,096, and their positions stay 32-bit integers.
constexpr int kKvMostTokens = INT32_MAX - 4095;

struct KvArgs {
    const int32_t* table;   // [seqs, max_pages]
    const int32_t* kv_len;  // [seqs]
    const int32_t* q_start; // [seqs + 1]
    int64_t num_pages;
    int max_tokens;         // positions that the table has pages for
    int seqs, max_pages, tokens;
    int page_shift;         // log2(page_size)
    int kv_heads, head_dim;
};

inline KvArgs kv_args(const mnb_kv_cache* c, const mnb_kv_batch* b) {
    KvArgs a;
    a.table = b->page_table;
    a.kv_len = b->kv_len;
    a.q_start = b->q_start;
    a.num_pages = c->num_pages;
    a.page_shift = 0;
    while ((1 << a.page_shift) < c->page_size) ++a.page_shift;
    const int64_t most = (int64_t)b->max_pages << a.page_shift;
    a.max_tokens = most > kKvMostTokens ? kKvMostTokens : (int)most;
    a.seqs = b->seqs;
    a.max_pages = b->max_pages;
    a.tokens = (int)b->tokens;
    a.kv_heads = c->kv_heads;
    a.head_dim = c->head_dim;
    return a;
}

// Work items of a sequence are numbered without a prefix sum over the batch:
// sequence s owns the items from first_item(s) = (q_start[s] * mul >> shift) +
// extra * s on.  The floor of the difference of two sums is at most one below
// the difference of the floors, so a sequence of n tokens always owns at least
// floor(n * mul / 2^shift) + extra items: with extra = 1 enough for its groups of
// 2^shift rows (mul rows a token), with extra = 2, mul = 1 and shift = 4 for the aligned
// blocks of 16 positions it touches (the first and the last partly).  Surplus items find
// nothing to do.
struct KvSplit {
    int mul, shift, extra;
};

__host__ __device__ inline int64_t kv_items(int64_t tokens, int seqs, KvSplit k) {
    return ((tokens * k.mul) >> k.shift) + (int64_t)k.extra * seqs;
}

// One sequence of the batch: its length, and its tokens of this call: rows row0 .. row0 + n - 1
// are the positions len - n .. len - 1.  The first ones may lie before 0, and the last ones past
// the table: positions from max_tokens on have no page, whatever the length says.
struct KvSeq {
    int s, len, row0, n;
};

__device__ __forceinline__ KvSeq kv_sequence(const KvArgs& a, int s, int q0, int q1, int l) {
    return {s, max(l, 0), q0, q1 > q0 ? min(q1 - q0, a.tokens) : 0};
}

__device__ __forceinline__ KvSeq kv_sequence(const KvArgs& a, int s) {
    return kv_sequence(a, s, a.q_start[s], a.q_start[s + 1], a.kv_len[s]);
}

// The sequence that owns item `u`, and its first item: a 32-way search by the whole warp (two
// rounds of loads up to 1024 sequences).  The last round's lanes hold single sequences, and
// load all there is to know of them at once: loads one behind the other are what a
// small call consists of.
__device__ __forceinline__ KvSeq kv_find_seq(const KvArgs& a, int64_t u, KvSplit k, int64_t* first) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.seqs;
    for (;;) {
        const int step = (hi - lo + 31) >> 5;
        const int s = lo + lane * step;
        int64_t at = INT64_MAX;
        int q0 = 0, q1 = 0, l = 0;
        if (s < hi) {
            q0 = a.q_start[s];
            if (step == 1) {
                q1 = a.q_start[s + 1];
                l = a.kv_len[s];
            }
            at = kv_items(q0, s, k);
        }
        const unsigned le = __ballot_sync(0xffffffffu, at <= u);
        const int last = le ? 31 - __clz(le) : 0;  // the first item of `lo` is never past u
        if (step == 1) {
            *first = __shfl_sync(0xffffffffu, at, last);
            return kv_sequence(a, lo + last, __shfl_sync(0xffffffffu, q0, last), __shfl_sync(0xffffffffu, q1, last),
                               __shfl_sync(0xffffffffu, l, last));
        }
        lo += last * step;
        hi = min(hi, lo + step);
    }
}

// The u-th longest sequence of up to kKvSortMost, by length in steps of 128 tokens, ties by number.
// The whole warp, one bit of the wanted length at a time.
constexpr int kKvSortMost = 256;
__device__ __forceinline__ int kv_by_length(const KvArgs& a, int u) {
    constexpr int kEach = kKvSortMost / 32;
    const int lane = threadIdx.x & 31;
    int len[kEach], most = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = i * 32 + lane;
        len[i] = s < a.seqs ? max(a.kv_len[s], 0) >> 7 : -1;
        most = max(most, len[i]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    auto count = [&](int t) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) n += len[i] >= t;
        return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
    };
    int t = 0;  // the length of the u-th: the largest that more than u sequences reach
    for (int bit = 31 - __clz(most | 1); bit >= 0; --bit)
        if (count(t | (1 << bit)) > u) t |= 1 << bit;
    int left = u - count(t + 1);
    int found = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const unsigned same = __ballot_sync(0xffffffffu, len[i] == t);
        const int n = __popc(same);
        const unsigned it = __ballot_sync(0xffffffffu, len[i] == t && __popc(same & ((1u << lane) - 1u)) == left);
        if (left >= 0 && left < n) found = i * 32 + __ffs(it) - 1;
        left -= n;
    }
    return found;
}

// Page of position `pos` (below max_tokens) of sequence s, or -1.
__device__ __forceinline__ int kv_page(const KvArgs& a, int s, int pos) {
    const int p = a.table[(int64_t)s * a.max_pages + (pos >> a.page_shift)];
    return p >= 0 && p < a.num_pages ? p : -1;
}

}  // namespace mnb
