// attn_common.cuh -- what the attention kernels share: the arguments of a call, the tiles of
// query rows, and the codes' unpacking.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kv_batch.cuh"
#include "mnb_internal.h"

namespace mnb {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

struct AttnArgs {
    KvArgs b;
    const uint8_t *K, *V;
    const float *Ks, *Vs;
    const __half* Q;
    __half* out;
    float* lse;          // [tokens, q_heads] or nullptr
    int64_t q_stride, out_stride;
    int q_heads, group;  // group: query heads of a kv head
    float scale_log2;    // scale * log2(e)
    int window;
    int single;          // every sequence has at most one row tile: tile u is sequence u's
    int chunk, splits;   // keys of a CTA, CTAs of a row tile
    int by_length;       // split kernel: tile u is that of the u-th longest sequence
    int cluster;         // split kernel: the CTAs of a row tile are a cluster, which joins the chunks
    int64_t skip_rows;   // prompt kernel: sequences with at most so many rows are the split kernel's
    int64_t most_rows;   // split kernel: those with more are the prompt kernel's
    float* part;         // [tokens * q_heads, splits, head_dim] (splits > 1)
    float* ml;           // [tokens * q_heads, splits, 2]: maximum of w, denominator
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr uint32_t kBias = 0x64806480u;  // half2(1024 + 128)

// Two codes (bytes `sel` of w) as exact FP16 integers q - 128.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_half2(uint32_t w) {
    return hsub2_rn(prmt(w, 0x64646464u, SEL), kBias);
}

// The rows of one tile: sequence, and the tile's first row among the sequence's
// n * group rows; false where the work item has no rows.
struct Tile {
    int s, len, n, r0;
    int64_t row0;  // token row of the sequence's first token of the call
};

__device__ __forceinline__ bool find_tile(const AttnArgs& a, int64_t u, int row_shift, Tile& t) {
    int64_t first = u;
    const KvSeq q = a.single ? kv_sequence(a.b, (int)u) : kv_find_seq(a.b, u, {a.group, row_shift, 1}, &first);
    t.s = q.s;
    t.len = q.len;
    t.n = q.n;
    t.row0 = q.row0;
    const int64_t r0 = (u - first) << row_shift;
    if (r0 < 0 || r0 >= (int64_t)t.n * a.group) return false;
    t.r0 = (int)r0;
    return true;
}

// First position that a token at `pos` (before 0, too) sees; any window, the largest int among them.
__device__ __forceinline__ int window_start(const AttnArgs& a, int pos) {
    return a.window > 0 ? max(max(pos, 0) - a.window + 1, 0) : 0;
}

constexpr int kPromptTile = 128;  // rows of one tile of the prompt kernel (attn_prompt.cu)
cudaError_t attn_prompt_prepare();
// row_tiles: 1 or 2 tiles a CTA; units: its row groups (kv_items)
cudaError_t attn_prompt_launch(const AttnArgs& a, int row_tiles, int64_t units, unsigned int* status, cudaStream_t st);

}  // namespace mnb
