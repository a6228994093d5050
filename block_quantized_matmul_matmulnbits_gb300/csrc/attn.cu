// attn.cu -- causal attention over the 8-bit key/value cache (mnb_attn).
//
// Per query row, with codes k_jd, v_jd (exact integers after subtracting 128)
// and one scale a block of 16 tokens:
//     s_j = scale * ks_b * sum_d q_d k_jd,     o = sum_j e^(s_j - m) vs_b v_j / sum_j e^(s_j - m)
// in one pass over the keys with a running maximum.
//
//  * The value scale goes into the exponent: w_j = s_j log2(e) + log2(vs_b), and
//    the running maximum is that of w.  The second product's left operand is then
//    2^(w_j - max w) <= 1 whatever the value scales are, so its FP16 rounding
//    (2^-11 of each term) never meets FP16's subnormals at the large end; the
//    denominator takes each block's sum times 1 / vs_b, in binary32.
//  * Codes become FP16 integers (1024 + q, then - 1152): both products take them
//    exactly, with binary32 accumulation (mma.sync m16n8k16).
//  * 16 query rows are one MMA row tile: consecutive (token, head of the kv
//    head's group) pairs, so the heads that share a kv head share its bytes.
//
// attn_split_kernel: a CTA of four warps takes one row tile, one kv head and
// `chunk` keys.  Each warp walks its own blocks of 16 keys (4 KB of codes at head_dim
// 128) through a ring of cp.async copies of its own, so nothing in the loop
// waits on another warp; the warps' results are joined once at the end, and the
// chunks' by attn_join_kernel where a row tile has more than one.  The codes are
// stored with their 16-byte chunks permuted by the row, so that both products'
// operand reads are free of bank conflicts.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_batch.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kRows = 16;     // query rows of a tile
constexpr int kWarps = 4;
constexpr int kStages = 4;    // blocks of 16 keys in a warp's ring
constexpr int kCtasPerSm = 3;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

constexpr uint32_t kBias = 0x64806480u;  // half2(1024 + 128)

// Two codes (bytes `sel` of w) as exact FP16 integers q - 128.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_half2(uint32_t w) {
    return hsub2_rn(prmt(w, 0x64646464u, SEL), kBias);
}

// Byte offset of 16-byte chunk c of row r in a block of 16 rows of D codes.
template <int D>
__device__ __forceinline__ uint32_t block_off(int r, int c) {
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The rows of one tile: sequence, and the tile's first row among the sequence's
// n * group rows; false where the work item has no rows.
struct Tile {
    int s, len, n, r0;
    int64_t row0;  // token row of the sequence's first token of the call
};

__device__ __forceinline__ bool find_tile(const AttnArgs& a, int64_t u, Tile& t) {
    int64_t first = u;
    t.s = a.single ? (int)u : kv_find_seq(a.b, u, a.group, 1, &first);
    int row0;
    kv_sequence(a.b, t.s, &t.len, &row0, &t.n);
    t.row0 = row0;
    const int64_t r0 = (u - first) * kRows;
    if (r0 < 0 || r0 >= (int64_t)t.n * a.group) return false;
    t.r0 = (int)r0;
    return true;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) attn_split_kernel(const AttnArgs a) {
    constexpr int KS = D / 16;           // k-steps of the first product
    constexpr int NN = D / 8;            // column tiles of the second
    constexpr int kBlockBytes = kKvBlock * D;
    constexpr int kStageBytes = 2 * kBlockBytes;
    constexpr int kCopies = kBlockBytes / 16 / 32;  // 16-byte copies a lane, keys or values
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    pdl_launch_dependents();

    Tile tl;
    if (!find_tile(a, blockIdx.x, tl)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int head = blockIdx.y, split = blockIdx.z;
    const int rows = (int)min((int64_t)tl.n * a.group - tl.r0, (int64_t)kRows);
    const int first = tl.len - tl.n;  // position of the call's first token

    // this lane's two rows: what they see is [lo, hi)
    int hi[2], lo[2];
    int64_t qoff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tl.r0 + g + 8 * i;
        const int tok = r / a.group;
        const int64_t row = tl.row0 + tok;
        const bool ok = g + 8 * i < rows && row >= 0 && row < a.b.tokens;
        const int pos = first + tok;
        hi[i] = ok ? max(pos + 1, 0) : 0;
        lo[i] = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
        qoff[i] = ok ? row * a.q_stride + (int64_t)(head * a.group + (r - tok * a.group)) * D : -1;
    }
    // the tile: its last token sees furthest, its first one starts furthest back
    const int tok_a = tl.r0 / a.group, tok_b = (tl.r0 + rows - 1) / a.group;
    const int hi_t = max(first + tok_b + 1, 0);
    const int lo_t = a.window > 0 ? max(first + tok_a - a.window + 1, 0) : 0;
    const int64_t begin64 = (int64_t)(lo_t & ~(kKvBlock - 1)) + (int64_t)split * a.chunk;
    const int begin = (int)min(begin64, (int64_t)hi_t);
    // the last chunk takes what is left, however long
    const int end = split == a.splits - 1 ? hi_t : (int)min(begin64 + a.chunk, (int64_t)hi_t);
    const int nblk = (end - begin + kKvBlock - 1) / kKvBlock;
    const int mine = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;
    // blocks that every row of the tile sees wholly need no mask
    const int all_hi = max(first + tok_a + 1, 0);
    const int all_lo = a.window > 0 ? max(first + tok_b - a.window + 1, 0) : 0;

    uint32_t qf[KS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4* src = reinterpret_cast<const uint4*>(a.Q + (qoff[i] < 0 ? 0 : qoff[i]) + t * (D / 4));
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            const uint4 v = qoff[i] < 0 || mine == 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + j);
            qf[2 * j][i] = v.x;
            qf[2 * j][2 + i] = v.y;
            qf[2 * j + 1][i] = v.z;
            qf[2 * j + 1][2 + i] = v.w;
        }
    }

    float o[NN][4];
#pragma unroll
    for (int j = 0; j < NN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * kStageBytes);
    // Where this warp's blocks lie, 32 blocks at a time, one a lane: the row of the
    // cache (-1: no such page) and the two scales; `next` is loaded while `cur` is used.
    const int pmask = (1 << a.b.page_shift) - 1;
    auto block_pos = [&](int i) { return begin + (warp + i * kWarps) * kKvBlock; };
    auto load_page = [&](int base) { return base + lane < mine ? kv_page(a.b, tl.s, block_pos(base + lane)) : -1; };
    auto slot_of = [&](int page, int base) {
        return page < 0 ? (int64_t)-1
                        : (((int64_t)page * a.b.kv_heads + head) << a.b.page_shift) + (block_pos(base + lane) & pmask);
    };
    auto load_scales = [&](int64_t slot, float& ks, float& vs) {
        ks = slot < 0 ? 0.f : __ldg(a.Ks + (slot >> 4));
        vs = slot < 0 ? 1.f : __ldg(a.Vs + (slot >> 4));
    };
    int64_t slot_cur = slot_of(load_page(0), 0), slot_nxt = -1;
    int page_nxt = -1;
    float ks_cur, vs_cur, ks_nxt = 0.f, vs_nxt = 1.f;
    load_scales(slot_cur, ks_cur, vs_cur);
    auto issue = [&](int i, int base) {  // block i of this warp into its ring; one copy group, maybe empty
        if (i < mine) {
            const int64_t slot = __shfl_sync(0xffffffffu, i - base < 32 ? slot_cur : slot_nxt, i & 31);
            if (slot >= 0) {
                const uint32_t dst = ring + (uint32_t)((i % kStages) * kStageBytes);
                const uint8_t* k = a.K + slot * D + lane * 16;
                const uint8_t* v = a.V + slot * D + lane * 16;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    const int id = lane + 32 * c;
                    const uint32_t off = block_off<D>(id / (D / 16), id % (D / 16));
                    cp_async16(dst + off, k + 512 * c);
                    cp_async16(dst + kBlockBytes + off, v + 512 * c);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, 0);

    for (int i = 0; i < mine; ++i) {
        const int base = i & ~31;
        if ((i & 31) == 0) {
            if (i > 0) {
                slot_cur = slot_nxt;
                ks_cur = ks_nxt;
                vs_cur = vs_nxt;
            }
            page_nxt = load_page(base + 32);
        } else if ((i & 31) == 8) {  // the pages have arrived long since
            slot_nxt = slot_of(page_nxt, base + 32);
            load_scales(slot_nxt, ks_nxt, vs_nxt);
        }
        issue(i + kStages - 1, base);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint32_t kb = ring + (uint32_t)((i % kStages) * kStageBytes), vb = kb + kBlockBytes;
        const float ks = __shfl_sync(0xffffffffu, ks_cur, i & 31) * a.scale_log2;
        const float vs0 = __shfl_sync(0xffffffffu, vs_cur, i & 31);
        const bool here = __shfl_sync(0xffffffffu, slot_cur >= 0 ? 1 : 0, i & 31) != 0;
        // A scale of zero has codes of zero value only: any scale gives the same products.
        // 2^-60 lies below every other scale (2^-31), so it never lifts the maximum.
        const float vs = vs0 == 0.f ? 8.67361738e-19f : vs0;
        const float lv = __log2f(vs), ivs = __frcp_rn(vs);

        // S = Q K^T: columns 2t, 2t + 1 of the two column tiles are keys 2t, 2t + 1 (+ 8)
        float sc[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[KS];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const uint4 v = lds128(kb + block_off<D>(g + 8 * h, t * (D / 64) + c));
                w[4 * c] = v.x;
                w[4 * c + 1] = v.y;
                w[4 * c + 2] = v.z;
                w[4 * c + 3] = v.w;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t b0 = codes_half2<0x4140u>(w[j]), b1 = codes_half2<0x4342u>(w[j]);
                if (j == 0)
                    mma_16816_z(sc[h], qf[j][0], qf[j][1], qf[j][2], qf[j][3], b0, b1);
                else
                    mma_16816(sc[h], qf[j][0], qf[j][1], qf[j][2], qf[j][3], b0, b1);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[h][c] = fmaf(sc[h][c], ks, lv);
        const int p0 = block_pos(i);
        if (!here || p0 < all_lo || p0 + kKvBlock > all_hi) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int j = p0 + 8 * h + 2 * t + (c & 1), r = c >> 1;
                    if (!here || j >= hi[r] || j < lo[r]) sc[h][c] = -INFINITY;
                }
        }
        float f[2], mu[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float x = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            x = fmaxf(x, m[r]);
            mu[r] = x == -INFINITY ? 0.f : x;  // a row that has seen nothing yet
            f[r] = ex2(m[r] - mu[r]);
            m[r] = x;
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < NN; ++j) {
                o[j][0] *= f[0];
                o[j][1] *= f[0];
                o[j][2] *= f[1];
                o[j][3] *= f[1];
            }
            l[0] *= f[0];
            l[1] *= f[1];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float p = ex2(sc[h][2 * r + c] - mu[r]);
                    sc[h][2 * r + c] = p;
                    sum += p;
                }
            if (sum != 0.f) l[r] = fmaf(sum, ivs, l[r]);  // a block hidden from the row may have any scale
        }
        const uint32_t a0 = pack_half2(sc[0][0], sc[0][1]), a1 = pack_half2(sc[0][2], sc[0][3]);
        const uint32_t a2 = pack_half2(sc[1][0], sc[1][1]), a3 = pack_half2(sc[1][2], sc[1][3]);

        // O += P V: lane (g, t) holds the codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 at
        // d = (D / 8) g + nn, column tile nn's column g
        uint32_t v[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 128) {
                const uint4 x = lds128(vb + block_off<D>(row, g));
                v[r][0] = x.x;
                v[r][1] = x.y;
                v[r][2] = x.z;
                v[r][3] = x.w;
            } else {
                const uint2 x = lds64(vb + block_off<D>(row, g >> 1) + (uint32_t)((g & 1) * 8));
                v[r][0] = x.x;
                v[r][1] = x.y;
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            // the two keys of a pair side by side: bytes (d, d, d + 1, d + 1)
            const uint32_t x0 = prmt(v[0][w], v[1][w], 0x5140u), x1 = prmt(v[0][w], v[1][w], 0x7362u);
            const uint32_t y0 = prmt(v[2][w], v[3][w], 0x5140u), y1 = prmt(v[2][w], v[3][w], 0x7362u);
            mma_16816(o[4 * w], a0, a1, a2, a3, codes_half2<0x4140u>(x0), codes_half2<0x4140u>(y0));
            mma_16816(o[4 * w + 1], a0, a1, a2, a3, codes_half2<0x4342u>(x0), codes_half2<0x4342u>(y0));
            mma_16816(o[4 * w + 2], a0, a1, a2, a3, codes_half2<0x4140u>(x1), codes_half2<0x4140u>(y1));
            mma_16816(o[4 * w + 3], a0, a1, a2, a3, codes_half2<0x4342u>(x1), codes_half2<0x4342u>(y1));
        }
        __syncwarp();  // the stage is read before it is filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            s_m[warp][g + 8 * r] = m[r];
            s_l[warp][g + 8 * r] = l[r];
        }
    }
    __syncthreads();  // also: every ring is free
    constexpr int kPitch = D + 4;
    float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][kRows][kPitch]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][row]);
        const float fac = ex2(m[r] - (mm == -INFINITY ? 0.f : mm));
        // d = (D / 4) t + nn and (D / 4) t + D / 8 + nn
        float* dst = s_o + (warp * kRows + row) * kPitch + t * (D / 4);
#pragma unroll
        for (int j = 0; j < NN; j += 4) {
            *reinterpret_cast<float4*>(dst + j) = make_float4(o[j][2 * r] * fac, o[j + 1][2 * r] * fac,
                                                              o[j + 2][2 * r] * fac, o[j + 3][2 * r] * fac);
            *reinterpret_cast<float4*>(dst + NN + j) =
                make_float4(o[j][2 * r + 1] * fac, o[j + 1][2 * r + 1] * fac, o[j + 2][2 * r + 1] * fac,
                            o[j + 3][2 * r + 1] * fac);
        }
    }
    __syncthreads();
    // eight threads a row, D / 8 values each (interleaved by four)
    const int row = threadIdx.x >> 3, part = threadIdx.x & 7;
    if (row >= rows) return;
    const int r = tl.r0 + row, tok = r / a.group;
    const int64_t trow = tl.row0 + tok;
    if (trow < 0 || trow >= a.b.tokens) return;
    const int qh = head * a.group + (r - tok * a.group);
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][row]);
    const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ll += s_l[w][row] * ex2(s_m[w][row] - mu);
    const int64_t orow = trow * a.q_heads + qh;
    const float inv = a.splits > 1 ? 1.f : (ll == 0.f ? 0.f : __fdiv_rn(1.f, ll));
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const int d = (c * 8 + part) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kRows + row) * kPitch + d);
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
        }
        if (a.splits > 1)
            *reinterpret_cast<float4*>(a.part + (orow * a.splits + split) * D + d) = sum;
        else
            *reinterpret_cast<uint2*>(a.out + trow * a.out_stride + (int64_t)qh * D + d) =
                make_uint2(pack_half2(sum.x * inv, sum.y * inv), pack_half2(sum.z * inv, sum.w * inv));
    }
    if (part == 0) {
        if (a.splits > 1)
            *reinterpret_cast<float2*>(a.ml + (orow * a.splits + split) * 2) = make_float2(mm, ll);
        else if (a.lse)
            a.lse[orow] = ll == 0.f ? -INFINITY : (mu + log2f(ll)) * kLn2;
    }
}

// The chunks of a row joined in their order: out = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c.
// One warp a row (token, query head).
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    pdl_wait();
    if (row >= (int64_t)a.b.tokens * a.q_heads) return;
    const float2* ml = reinterpret_cast<const float2*>(a.ml) + row * a.splits;
    float mm = -INFINITY;
    for (int c = lane; c < a.splits; c += 32) mm = fmaxf(mm, ml[c].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
    const float mu = mm == -INFINITY ? 0.f : mm;
    constexpr int V = D / 32;  // values a lane
    float acc[V], ll = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    const float* part = a.part + row * a.splits * D + lane * V;
    for (int c = 0; c < a.splits; ++c) {
        const float2 x = ml[c];
        const float f = ex2(x.x - mu);
        ll = fmaf(x.y, f, ll);
        if (x.x == -INFINITY && x.y == 0.f) continue;  // a chunk with nothing to see: its sums are zeros
        if constexpr (V == 4) {
            const float4 p = *reinterpret_cast<const float4*>(part + (int64_t)c * D);
            acc[0] = fmaf(p.x, f, acc[0]);
            acc[1] = fmaf(p.y, f, acc[1]);
            acc[2] = fmaf(p.z, f, acc[2]);
            acc[3] = fmaf(p.w, f, acc[3]);
        } else {
            const float2 p = *reinterpret_cast<const float2*>(part + (int64_t)c * D);
            acc[0] = fmaf(p.x, f, acc[0]);
            acc[1] = fmaf(p.y, f, acc[1]);
        }
    }
    const float inv = ll == 0.f ? 0.f : __fdiv_rn(1.f, ll);
    const int64_t tok = row / a.q_heads;
    const int qh = (int)(row - tok * a.q_heads);
    __half* dst = a.out + tok * a.out_stride + (int64_t)qh * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_half2(acc[0] * inv, acc[1] * inv), pack_half2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_half2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && a.lse) a.lse[row] = ll == 0.f ? -INFINITY : (mu + log2f(ll)) * kLn2;
}

constexpr int split_smem(int D) {
    const int ring = kWarps * kStages * 2 * kKvBlock * D, join = kWarps * kRows * (D + 4) * 4;
    return ring > join ? ring : join;
}

struct AttnPlan {
    int64_t units;
    int single, chunk, splits;
    int64_t ws_bytes;
};

// How the keys are dealt out: about two CTAs' worth of work for every CTA slot of
// the GPU, in whole rounds of the four warps, at least 128 keys a CTA.
int attn_plan(const mnb_kv_cache* c, const mnb_kv_batch* b, int q_heads, int window, int sms, AttnPlan* p) {
    const int G = q_heads / c->kv_heads;
    p->single = (int64_t)b->max_new * G <= kRows;
    p->units = p->single ? b->seqs : kv_items(b->tokens, b->seqs, G, 1);
    if (p->units > INT32_MAX) return MNB_ERR_UNSUPPORTED;
    int64_t keys = b->max_len;
    // a tile's rows lie kRows / G + 1 tokens apart at most; its range starts at a block's start
    if (window > 0) keys = keys < (int64_t)window + kRows / G + 1 + kKvBlock ? keys : (int64_t)window + kRows / G + 1 + kKvBlock;
    if (keys < 1) keys = 1;
    const int64_t want = (p->units * c->kv_heads * keys) / ((int64_t)sms * kCtasPerSm * 2) + 1;
    const int64_t round = kWarps * kKvBlock;
    int64_t chunk = (want + round - 1) / round * round;
    if (chunk < 2 * round) chunk = 2 * round;
    p->splits = (int)((keys + chunk - 1) / chunk);
    if (p->splits == 1) chunk = (keys + kKvBlock - 1) / kKvBlock * kKvBlock;
    p->chunk = (int)(chunk < INT32_MAX - 64 ? chunk : INT32_MAX - 63);
    p->ws_bytes = p->splits > 1 ? (int64_t)b->tokens * q_heads * p->splits * (c->head_dim + 2) * 4 : 0;
    return MNB_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D>
cudaError_t launch(const AttnArgs& a, const AttnPlan& p, cudaStream_t st) {
    attn_split_kernel<D><<<dim3((unsigned)p.units, (unsigned)a.b.kv_heads, (unsigned)p.splits), kWarps * 32,
                           split_smem(D), st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.b.tokens * a.q_heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, a);
}

// The checks mnb_attn and mnb_attn_workspace share.
int attn_check(const mnb_kv_cache* c, const mnb_kv_batch* b, int q_heads, int window, bool* empty) {
    const int rc = kv_check(c, b, empty);
    if (rc != MNB_OK) return rc;
    if (q_heads <= 0 || window < 0) return MNB_ERR_ARG;
    if (q_heads % c->kv_heads != 0 || q_heads > 65535) return MNB_ERR_UNSUPPORTED;
    if ((int64_t)b->tokens * q_heads > (int64_t)1 << 40) return MNB_ERR_UNSUPPORTED;
    return MNB_OK;
}

}  // namespace

cudaError_t attn_prepare() {
    cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, split_smem(64));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_split_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, split_smem(128));
}

}  // namespace mnb

extern "C" int64_t mnb_attn_workspace(const mnb_kv_cache* cache, const mnb_kv_batch* batch, int32_t q_heads,
                                      int32_t window, int32_t sm_count) {
    bool empty;
    int rc = mnb::attn_check(cache, batch, q_heads, window, &empty);
    if (rc != MNB_OK) return rc;
    if (empty) return 0;
    int sms = sm_count;
    unsigned int* status;
    if (sms <= 0 && (rc = mnb::device_ready(&sms, &status)) != MNB_OK) return rc;
    mnb::AttnPlan p;
    rc = mnb::attn_plan(cache, batch, q_heads, window, sms, &p);
    return rc != MNB_OK ? rc : p.ws_bytes;
}

extern "C" int mnb_attn(const mnb_kv_cache* cache, const mnb_kv_batch* batch, const void* Q, int64_t q_stride,
                        int32_t q_heads, float scale, int32_t window, void* out, int64_t out_stride, float* lse,
                        void* ws, int64_t ws_bytes, void* stream) {
    bool empty;
    int rc = mnb::attn_check(cache, batch, q_heads, window, &empty);
    if (rc != MNB_OK) return rc;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    if (q_stride < width || out_stride < width || ws_bytes < 0) return MNB_ERR_ARG;
    if (q_stride % 8 != 0 || out_stride % 8 != 0) return MNB_ERR_ALIGN;
    if (empty) return MNB_OK;
    if (!Q || !out) return MNB_ERR_ARG;
    if (!mnb::aligned(Q, 16) || !mnb::aligned(out, 16) || !mnb::aligned(lse, 4) || !mnb::aligned(ws, 16))
        return MNB_ERR_ALIGN;
    int sms;
    unsigned int* status;
    rc = mnb::device_ready(&sms, &status);
    if (rc != MNB_OK) return rc;
    mnb::AttnPlan p;
    rc = mnb::attn_plan(cache, batch, q_heads, window, sms, &p);
    if (rc != MNB_OK) return rc;
    if (p.ws_bytes > 0 && (!ws || ws_bytes < p.ws_bytes)) return MNB_ERR_ARG;
    mnb::AttnArgs a;
    a.b = mnb::kv_args(cache, batch);
    a.K = static_cast<const uint8_t*>(cache->K);
    a.V = static_cast<const uint8_t*>(cache->V);
    a.Ks = static_cast<const float*>(cache->K_scales);
    a.Vs = static_cast<const float*>(cache->V_scales);
    a.Q = static_cast<const __half*>(Q);
    a.out = static_cast<__half*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale_log2 = scale * mnb::kLog2e;
    a.window = window;
    a.single = p.single;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.part = static_cast<float*>(ws);
    a.ml = a.part ? a.part + batch->tokens * (int64_t)q_heads * p.splits * cache->head_dim : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->head_dim == 64 ? mnb::launch<64>(a, p, st) : mnb::launch<128>(a, p, st);
    return e == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
