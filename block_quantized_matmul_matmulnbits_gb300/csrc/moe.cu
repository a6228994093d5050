// moe.cu -- a mixture-of-experts layer of block-quantized gated MLPs for up to 16 tokens
// (mnb_moe): three kernels, each started before the one ahead of it ends.
//
//   router   logits x . r_e, one CTA an expert and four tokens.  Which expert comes first decides the
//            output, so the sums are held in two FP32 words each (products of FP16 are exact).
//   up       every CTA picks the experts again from the logits (a warp a token), makes the
//            list of (expert, some of its tokens) and takes units of 32 features of one
//            item: gate and up rows, a warp 16 rows by a slice of the inputs.
//   down     a cluster takes 16 outputs over all items, so the sum over experts stays in it.
//
// Every warp streams its own weights and inputs into a ring of steps in shared memory (cp.async: prefetched in
// registers, 16 warps an SM waited for loads half of the time, since a short load's scoreboard is the
// long ones' too).  A lane takes 16 bytes of codes a row: a quad's lanes hold four neighbouring blocks of 32 inputs.  A lane takes the zero point of its own
// block off (exact in FP16) and the rows go to the MMA (m16n8k16) as its left operand.
// A step's columns are two tokens by the quad's four blocks: the right operand is zero
// but where a column's block is the lane's own, so each column sums one block of one
// token, exact codes times FP16 inputs in FP32, and the block's scale multiplies its sum in FP32.
// No code is rounded and no sum over K is needed for the zero points.  Two tokens a
// step use a quarter of the MMA's work; an expert of a few tokens' step has one or two.
//
// The inputs lie in the workspace as the MMA takes them (router and up kernel write them so): 256 bytes
// a step, first the quad's first quarter blocks and so on, each in the order of the codes, a
// row of zeros for the lanes that have none, zeros up to a whole step.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_batch.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kTokens = MNB_MOE_MAX_TOKENS;
constexpr int kMaxExperts = 256;
constexpr int kMaxTop = 16;
constexpr int kMostItem = 8;               // tokens of an item, at most
constexpr int kMaxItems = kTokens * kMaxTop;
constexpr int kTile = 32;                  // features of a unit of the up kernel

struct MoeWeight {
    const uint8_t* q;
    const __half* s;
    const uint8_t* z;
};

// The items of a call: an expert and some of its tokens each.
struct MoeTable {
    int count;
    uint16_t expert[kMaxItems];
    uint16_t n[kMaxItems];                 // tokens of the item
    uint16_t row[kMaxItems][kMostItem];    // token | slot << 8
};

struct MoeArgs {
    int hidden, inter, experts, top_k, tokens, normalize, bits;
    const __half* x;
    const __half* router;
    MoeWeight up, down;
    int item;             // tokens of an item
    double* logits;       // [tokens, experts]
    MoeTable* table;      // the items, for the down kernel
    char* xs;             // [tokens + 1] rows of x, the last of zeros
    char* h;              // [tokens * top_k + 1] rows of silu(gate) up / 2^e, e of each 32; the last of zeros
    float* he;            // [tokens * top_k, 4 steps]: weight * 2^e
    __half* y;
    int32_t* ids;
    float* weights;
};

// ---- router ---------------------------------------------------------------

constexpr int kRouterThreads = 128;
constexpr int kRouterTokens = 4;

// s + e = s + e + p, to about twice FP32's places (Knuth's two-sum).
__device__ __forceinline__ void add2(float& s, float& e, float p) {
    const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
    s = t;
}

// Bytes of a row of `cols` values as the MMA takes them.
__host__ __device__ __forceinline__ int64_t row_bytes(int cols) { return (int64_t)((cols + 127) >> 7) * 256; }

// Where eight values from 8 i on go, and in which order (4-bit codes: 0 4 1 5 2 6 3 7).
__device__ __forceinline__ int piece_at(int i) { return (i >> 4) * 256 + (i & 3) * 64 + ((i >> 2) & 3) * 16; }
__device__ __forceinline__ uint4 in_order(const uint4& v, int bits) {
    return bits == 8 ? v : make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u),
                                      prmt(v.y, v.w, 0x7632u));
}

__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a) {
    __shared__ double part[kRouterThreads / 32][kRouterTokens];
    const int tid = threadIdx.x, lane = tid & 31, e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
    pdl_wait();
    pdl_launch_dependents();
    const int n = min(a.tokens - t0, kRouterTokens), pieces = a.hidden >> 3;
    if (e == a.experts) {  // the inputs, once for all
        const int all = (int)(row_bytes(a.hidden) >> 4);
        for (int t = 0; t <= n; ++t) {
            if (t == n && blockIdx.y != 0) break;
            const int row = t == n ? a.tokens : t0 + t;
            for (int i = tid; i < all; i += kRouterThreads) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (t < n && i < pieces)
                    v = in_order(reinterpret_cast<const uint4*>(a.x + (int64_t)row * a.hidden)[i], a.bits);
                *reinterpret_cast<uint4*>(a.xs + row * row_bytes(a.hidden) + piece_at(i)) = v;
            }
        }
        if (blockIdx.y == 0)
            for (int i = tid; i < (int)(row_bytes(a.inter) >> 4); i += kRouterThreads)
                reinterpret_cast<uint4*>(a.h + (int64_t)a.tokens * a.top_k * row_bytes(a.inter))[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const uint4* r = reinterpret_cast<const uint4*>(a.router + (int64_t)e * a.hidden);
    float s[kRouterTokens] = {}, c[kRouterTokens] = {};
    for (int i = tid; i < pieces; i += kRouterThreads) {
        const uint4 w = r[i];
        const __half2* w2 = reinterpret_cast<const __half2*>(&w);
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t) {
            if (t >= n) break;
            const uint4 v = reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * a.hidden)[i];
            const __half2* v2 = reinterpret_cast<const __half2*>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(w2[j]), g = __half22float2(v2[j]);
                add2(s[t], c[t], __fmul_rn(f.x, g.x));
                add2(s[t], c[t], __fmul_rn(f.y, g.y));
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
        if (t >= n) break;
        double d = (double)s[t] + (double)c[t];
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
        if (lane == 0) part[tid >> 5][t] = d;
    }
    __syncthreads();
    if (tid < n) {
        double d = part[0][tid];
#pragma unroll
        for (int w = 1; w < kRouterThreads / 32; ++w) d += part[w][tid];
        a.logits[(int64_t)(t0 + tid) * a.experts + e] = d;
    }
}

// ---- the choice of experts, and the items ----------------------------------

struct MoeItems {
    MoeTable t;
    uint32_t mask[kMaxExperts];            // tokens of an expert
    uint16_t first[kMaxExperts];           // its first item
    int32_t sel[kTokens * kMaxTop];
    float weight[kTokens * kMaxTop];
};

__device__ __forceinline__ unsigned long long order64(double d) {
    if (d != d) return 1;  // NaN: below every number, still a choice
    const long long b = __double_as_longlong(d + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

__device__ __forceinline__ float exp_of(double d) {  // d <= 0, or NaN
    const float hi = (float)d;
    return expf(hi) * (1.f + (isfinite(hi) ? (float)(d - (double)hi) : 0.f));
}

// The top_k experts of a token, by the whole warp: the largest logit top_k times.
__device__ void moe_choose(const MoeArgs& a, int token, int32_t* sel, float* weight) {
    constexpr int kEach = kMaxExperts / 32;
    const int lane = threadIdx.x & 31;
    const double* l = a.logits + (int64_t)token * a.experts;
    unsigned long long key[kEach];
    double v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0;
        v[i] = 0.0;
        if (i * 32 >= a.experts) continue;
        if (e < a.experts) {
            v[i] = l[e];
            key[i] = order64(v[i]);
        }
    }
    double top = 0.0, mine = 0.0;
    for (int r = 0; r < a.top_k; ++r) {
        unsigned long long best = key[0];
        double bv = v[0];
        int be = lane;
#pragma unroll
        for (int i = 1; i < kEach; ++i) {
            if (i * 32 >= a.experts) break;
            if (key[i] > best) best = key[i], bv = v[i], be = i * 32 + lane;
        }
        const unsigned hi = (unsigned)(best >> 32), m = __reduce_max_sync(0xffffffffu, hi);
        const unsigned lo = hi == m ? (unsigned)best : 0u, m2 = __reduce_max_sync(0xffffffffu, lo);
        const int e = __reduce_min_sync(0xffffffffu, hi == m && lo == m2 ? be : INT32_MAX);
        const double chosen = __shfl_sync(0xffffffffu, bv, e & 31);
        if (r == 0) top = chosen;
        if (lane == r) {
            mine = chosen;
            sel[r] = e;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i * 32 >= a.experts) break;
            if (e == i * 32 + lane) key[i] = 0;
        }
    }
    float w = lane < a.top_k ? exp_of(mine - top) : 0.f, sum = 0.f;
    if (a.normalize) {
        sum = w;
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i * 32 >= a.experts) break;
            if (i * 32 + lane < a.experts) sum += exp_of(v[i] - top);
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane < a.top_k) weight[lane] = __fdiv_rn(w, sum);
}

// The items of the chosen experts (sel in place): by expert number, a.item tokens each. Whole CTA.
__device__ void moe_items(const MoeArgs& a, MoeItems& it) {
    const int tid = threadIdx.x, lane = tid & 31, picks = a.tokens * a.top_k;
    for (int e = tid; e < a.experts; e += blockDim.x) it.mask[e] = 0;
    __syncthreads();
    if (tid < picks) atomicOr(&it.mask[it.sel[tid]], 1u << (tid / a.top_k));
    __syncthreads();
    if (tid < 32) {
        int at = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            int n = e < a.experts ? __popc(it.mask[e]) : 0;
            const int items = (n + a.item - 1) / a.item;
            int run = items;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, run, d);
                if (lane >= d) run += o;
            }
            const int first = at + run - items;
            if (e < a.experts) it.first[e] = (uint16_t)first;
            for (int i = 0; i < items; ++i, n -= a.item) {
                it.t.expert[first + i] = (uint16_t)e;
                it.t.n[first + i] = (uint16_t)min(n, a.item);
            }
            at += __shfl_sync(0xffffffffu, run, 31);
        }
        if (lane == 0) it.t.count = at;
    }
    __syncthreads();
    if (tid < picks) {
        const int t = tid / a.top_k, e = it.sel[tid];
        const int at = __popc(it.mask[e] & ((1u << t) - 1u));
        it.t.row[it.first[e] + at / a.item][at % a.item] = (uint16_t)(t | (tid - t * a.top_k) << 8);
    }
    __syncthreads();
}

// ---- 16 rows of weights times an item's tokens -------------------------------

// Asynchronous copies into shared memory; `there` = false fills with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {  // read once: past L1
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A step in the ring: 16 rows by four blocks of codes (each lane's pieces behind one another's), scales [16][4], zero points
// [16][4], inputs (256 bytes a token), the tokens' factors [4].
template <int BITS, int NP>
struct Slot {
    static constexpr int kScales = 256 * BITS, kZeros = kScales + 128, kInputs = kZeros + 64,
                         kFactors = kInputs + NP * 512, kBytes = kFactors + NP * 32;
};

// Where a lane's copies of a tile come from, moved on step by step: its codes' block of row lane / 4 and of the one eight
// behind, two scales of row lane / 2, four zero points of row lane (lanes 0 to 15).
struct TilePtr {
    const uint8_t *q, *q8, *s, *z;
};

template <int BITS>
__device__ __forceinline__ TilePtr tile_at(const MoeWeight& w, int64_t row, int step, int nblk) {
    const int lane = threadIdx.x & 31;
    const uint8_t* q = w.q + ((row + (lane >> 2)) * nblk + step * 4 + (lane & 3)) * (4 * BITS);
    return {q, q + nblk * (32 * BITS),
            reinterpret_cast<const uint8_t*>(w.s + (row + (lane >> 1)) * nblk + step * 4 + (lane & 1) * 2),
            w.z + (w.z ? (row + (lane & 15)) * nblk + step * 4 : 0)};
}

// Copies of a step's weights; blocks past the row's end (`left` of them are there) are zeros.  words: rows of scales and zero
// points begin at a word, and all steps are whole.
template <int BITS, int NP>
__device__ __forceinline__ void copy_weights(uint32_t slot, TilePtr& p, bool words, int left) {
    using S = Slot<BITS, NP>;
    const int lane = threadIdx.x & 31;
    if (words) {
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) {
            copy16(slot + lane * 16 + i * 1024, p.q + i * 16, true);
            copy16(slot + lane * 16 + i * 1024 + 512, p.q8 + i * 16, true);
        }
        copy4(slot + S::kScales + lane * 4, p.s);
        if (p.z) copy4(slot + S::kZeros + (lane & 15) * 4, p.z);  // (twice the same)
    } else {
        const bool there = (lane & 3) < left;
        const int64_t back = there ? 0 : -(int64_t)(lane & 3) * (4 * BITS);  // a block that is there
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) {
            copy16(slot + lane * 16 + i * 1024, p.q + back + i * 16, there);
            copy16(slot + lane * 16 + i * 1024 + 512, p.q8 + back + i * 16, there);
        }
        const int b = (lane & 1) * 2;
        const __half* s = reinterpret_cast<const __half*>(p.s);
        const uint32_t lo = b < left ? __half_as_ushort(s[0]) : 0, hi = b + 1 < left ? __half_as_ushort(s[1]) : 0;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot + S::kScales + lane * 4), "r"(lo | hi << 16) : "memory");
        if (p.z && lane < 16) {
            uint32_t v = 0;
            for (int i = 0; i < 4 && i < left; ++i) v |= (uint32_t)p.z[i] << (8 * i);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot + S::kZeros + lane * 4), "r"(v) : "memory");
        }
    }
    p.q += 16 * BITS;
    p.q8 += 16 * BITS;
    p.s += 8;
    if (p.z) p.z += 4;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Eight codes less their zero point as FP16 (exact): c = 1024 + zp twice, d = -(64 + zp) twice.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t c, uint32_t d, uint32_t o[4]) {
    const uint32_t w8 = w >> 8;
    o[0] = hsub2_rn(lop3_and_or(w, 0x000F000Fu, kMagic1024x2), c);                   // codes 0, 4
    o[1] = hfma2_rn(lop3_and_or(w, 0x00F000F0u, kMagic1024x2), kSixteenthX2, d);     // 1, 5
    o[2] = hsub2_rn(lop3_and_or(w8, 0x000F000Fu, kMagic1024x2), c);                  // 2, 6
    o[3] = hfma2_rn(lop3_and_or(w8, 0x00F000F0u, kMagic1024x2), kSixteenthX2, d);    // 3, 7
}

__device__ __forceinline__ void codes8(uint32_t lo, uint32_t hi, uint32_t c, uint32_t o[4]) {
    o[0] = hsub2_rn(prmt(lo, 0x64646464u, 0x4140u), c);
    o[1] = hsub2_rn(prmt(lo, 0x64646464u, 0x4342u), c);
    o[2] = hsub2_rn(prmt(hi, 0x64646464u, 0x4140u), c);
    o[3] = hsub2_rn(prmt(hi, 0x64646464u, 0x4342u), c);
}

// Adds a step (four blocks of 16 rows) times 2 P tokens: y[p][0], y[p][1] are rows g and
// g + 8 of token 2 p + (lane & 3) / 2, blocks 2 (lane & 1) and the one behind it.  zeros: NP * 512 bytes of zeros, the inputs of
// lanes that have none: column g = lane / 4 is token g / 4, block g % 4, and only the lanes that hold that block have any.
template <int BITS, int NP, int P, bool FACTORS>
__device__ __forceinline__ void step_of(const uint8_t* slot, const uint8_t* zeros, bool zp, float (*y)[2]) {
    using S = Slot<BITS, NP>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t za = 1u << (BITS - 1), zb = za;
    if (zp) {
        za = slot[S::kZeros + lane];
        zb = slot[S::kZeros + 32 + lane];
    }
    const uint4* codes = reinterpret_cast<const uint4*>(slot) + lane;
    uint4 ra[BITS / 4], rb[BITS / 4];
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
        ra[i] = codes[i * 64];
        rb[i] = codes[i * 64 + 32];
    }
    const uint8_t* x = (g & 3) == t ? slot + S::kInputs + (g >> 2) * 256 + t * 16 : zeros;
    const uint32_t ca = kMagic1024x2 | za * 0x00010001u, cb = kMagic1024x2 | zb * 0x00010001u;
    const uint32_t da = hsub2_rn(kHalf960x2, ca), db = hsub2_rn(kHalf960x2, cb);
    float c[P][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t A[4], B[4];
        if (BITS == 4) {
            codes4(word(ra[0], j), ca, da, A);
            codes4(word(rb[0], j), cb, db, B);
        } else {
            constexpr int kHi = BITS / 4 - 1;
            codes8(word(ra[j / 2 * kHi], 2 * j % 4), word(ra[j / 2 * kHi], (2 * j + 1) % 4), ca, A);
            codes8(word(rb[j / 2 * kHi], 2 * j % 4), word(rb[j / 2 * kHi], (2 * j + 1) % 4), cb, B);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint4 v = *reinterpret_cast<const uint4*>(x + p * 512 + j * 64);
            if (j == 0)
                mma_16816_z(c[p], A[0], B[0], A[1], B[1], v.x, v.y);
            else
                mma_16816(c[p], A[0], B[0], A[1], B[1], v.x, v.y);
            mma_16816(c[p], A[2], B[2], A[3], B[3], v.z, v.w);
        }
    }
    // scales of the two blocks that this lane holds sums of
    const __half2* scales = reinterpret_cast<const __half2*>(slot + S::kScales + g * 8 + (t & 1) * 4);
    const float2 f0 = __half22float2(scales[0]), f1 = __half22float2(scales[16]);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (FACTORS) {
            const float2 f = *reinterpret_cast<const float2*>(slot + S::kFactors + (2 * p + (t >> 1)) * 16 + (t & 1) * 8);
            y[p][0] = fmaf(f0.y * f.y, c[p][1], fmaf(f0.x * f.x, c[p][0], y[p][0]));
            y[p][1] = fmaf(f1.y * f.y, c[p][3], fmaf(f1.x * f.x, c[p][2], y[p][1]));
        } else {
            y[p][0] = fmaf(f0.y, c[p][1], fmaf(f0.x, c[p][0], y[p][0]));
            y[p][1] = fmaf(f1.y, c[p][3], fmaf(f1.x, c[p][2], y[p][1]));
        }
    }
}

// The step for so many pairs (three are done as four): one branch, not one at every product.
template <int BITS, int NP, bool FACTORS>
__device__ __forceinline__ void do_step(const uint8_t* slot, const uint8_t* zeros, bool zp, int pairs, float (*y)[2]) {
    if (NP == 1 || pairs == 1)
        step_of<BITS, NP, 1, FACTORS>(slot, zeros, zp, y);
    else if (NP == 2 || pairs == 2)
        step_of<BITS, NP, (NP < 2 ? NP : 2), FACTORS>(slot, zeros, zp, y);
    else
        step_of<BITS, NP, NP, FACTORS>(slot, zeros, zp, y);
}

// ---- gate and up -------------------------------------------------------------

// Variants: NP, pairs of tokens of an item, and SLICES, warps that share a row's inputs; RING steps in shared memory.
template <int BITS, int NP, int SLICES, int RING, int CTAS>
__global__ void __launch_bounds__(SLICES * 128, CTAS) moe_up_kernel(const MoeArgs a) {
    using S = Slot<BITS, NP>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ MoeItems it;
    __shared__ float red[2][SLICES][4][16][2 * NP + 1];
    __shared__ uint4 zero[NP * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < NP * 32) zero[tid] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_launch_dependents();
    for (int t = warp; t < a.tokens; t += SLICES * 4)
        moe_choose(a, t, it.sel + t * a.top_k, it.weight + t * a.top_k);
    __syncthreads();
    if (blockIdx.x == 0 && tid < a.tokens * a.top_k) {
        if (a.ids) a.ids[tid] = it.sel[tid];
        if (a.weights) a.weights[tid] = it.weight[tid];
    }
    moe_items(a, it);
    if (blockIdx.x == 0) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(&it.t);
        for (int i = tid; i < (int)sizeof(MoeTable) / 4; i += SLICES * 128) reinterpret_cast<uint32_t*>(a.table)[i] = from[i];
    }

    const int nblk = a.hidden >> 5, steps = (nblk + 3) >> 2, tiles = a.inter / kTile;
    const int q = warp & 3, slice = warp >> 2;  // gate, gate + 16, up, up + 16; which part of the inputs
    const int s0 = steps * slice / SLICES, s1 = steps * (slice + 1) / SLICES;
    const int64_t pitch = row_bytes(a.hidden), hpitch = row_bytes(a.inter);
    const bool words = !(nblk & 3);
    // the CTA's units, one every gridDim.x: item and tile without a division each
    const int by_item = gridDim.x / tiles, by_tile = gridDim.x - by_item * tiles;
    struct Unit {
        int item, tile;
    };
    const Unit first = {(int)blockIdx.x / tiles, (int)blockIdx.x % tiles};
    auto next = [&](Unit& u) {
        u.item += by_item;
        u.tile += by_tile;
        if (u.tile >= tiles) u.tile -= tiles, ++u.item;
    };
    const int64_t row0 = (int64_t)(q >> 1) * a.inter + (q & 1) * 16;
    uint8_t* const own = ring + warp * (RING * S::kBytes);
    const uint32_t base = smem_u32(own);
    const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(zero);
    Unit lu = first;  // what is copied next
    int ls = s0, lpairs = 0;
    bool more = s0 < s1 && lu.item < it.t.count;
    uint32_t lslot = base;
    TilePtr lp;
    const char* lx[NP];
    auto aim = [&] {
        lp = tile_at<BITS>(a.up, (int64_t)it.t.expert[lu.item] * 2 * a.inter + row0 + lu.tile * kTile, s0, nblk);
        const int n = it.t.n[lu.item];
        lpairs = (n + 1) >> 1;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = 2 * p + (lane >> 4);
            lx[p] = a.xs + (i < n ? it.t.row[lu.item][i] & 255 : a.tokens) * pitch + s0 * 256 + (lane & 15) * 16;
        }
    };
    auto issue = [&] {
        if (more) {
            copy_weights<BITS, NP>(lslot, lp, words, nblk - ls * 4);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                if (p < lpairs) copy16_l1(lslot + S::kInputs + p * 512 + lane * 16, lx[p]);
                lx[p] += 256;
            }
            if (++ls == s1) {
                ls = s0;
                next(lu);
                more = lu.item < it.t.count;
                if (more) aim();
            }
        }
        copies_end();
        lslot = lslot == base + (RING - 1) * S::kBytes ? base : lslot + S::kBytes;
    };
    if (more) aim();
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) issue();
    int buf = 0;
    const uint8_t* slot = own;
    for (Unit u = first; u.item < it.t.count; next(u), buf ^= 1) {
        const int item = u.item, tile = u.tile, n = it.t.n[item], pairs = (n + 1) >> 1;
        float y[NP][2];
#pragma unroll
        for (int p = 0; p < NP; ++p) y[p][0] = y[p][1] = 0.f;
        for (int s = s0; s < s1; ++s) {
            copies_wait<RING - 2>();
            __syncwarp();  // everyone's copies are there, and the slot before is read
            issue();
            do_step<BITS, NP, false>(slot, zeros, a.up.z != nullptr, pairs, y);
            slot = slot == own + (RING - 1) * S::kBytes ? own : slot + S::kBytes;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (p >= pairs) break;
            const float v0 = y[p][0] + __shfl_xor_sync(0xffffffffu, y[p][0], 1);
            const float v1 = y[p][1] + __shfl_xor_sync(0xffffffffu, y[p][1], 1);
            if (!(lane & 1)) {
                red[buf][slice][q][lane >> 2][2 * p + ((lane & 3) >> 1)] = v0;
                red[buf][slice][q][(lane >> 2) + 8][2 * p + ((lane & 3) >> 1)] = v1;
            }
        }
        __syncthreads();
        for (int w = warp; w < n; w += SLICES * 4) {  // a warp a token, a lane a feature
            const int f = lane;
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int i = 0; i < SLICES; ++i) {
                gate += red[buf][i][f >> 4][f & 15][w];
                up += red[buf][i][2 + (f >> 4)][f & 15][w];
            }
            const float h = gate / (1.f + expf(-gate)) * up;
            float m = fabsf(h);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            // FP16 holds the block about its largest value, whatever that is: 2^e <= m < 2^(e + 1)
            uint32_t e = __float_as_uint(m) & 0x7F800000u;
            e = e == 0 || e >= 0x7F000000u ? 0x3F800000u : e;
            const int row = it.t.row[item][w], at = (row & 255) * a.top_k + (row >> 8);
            // feature f of the tile's block, as the MMA takes it
            char* to = a.h + at * hpitch + (tile >> 2) * 256 + (f >> 3) * 64 + (tile & 3) * 16;
            const int in = BITS == 8 ? f & 7 : (f & 3) * 2 + ((f >> 2) & 1);
            reinterpret_cast<__half*>(to)[in] = __float2half_rn(h * __uint_as_float(0x7F000000u - e));
            float* fe = a.he + (int64_t)at * ((tiles + 3) & ~3);
            if (lane == 0) fe[tile] = it.weight[at] * __uint_as_float(e);
            if (tile == tiles - 1)  // zeros up to a whole step
                for (int b = tiles; b < ((tiles + 3) & ~3); ++b) {
                    if (lane < 4)
                        *reinterpret_cast<uint4*>(a.h + at * hpitch + (b >> 2) * 256 + lane * 64 + (b & 3) * 16) =
                            make_uint4(0, 0, 0, 0);
                    if (lane == 0) fe[b] = 0.f;
                }
        }
    }
}

// ---- down ----------------------------------------------------------------------

constexpr int kDownWarps = 4;

template <int BITS, int NP, int RING, int CTAS>
__global__ void __launch_bounds__(kDownWarps * 32, CTAS) moe_down_kernel(const MoeArgs a) {
    using S = Slot<BITS, NP>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float acc[kDownWarps][kTokens][17];
    __shared__ uint4 zero[NP * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < NP * 32) zero[tid] = make_uint4(0, 0, 0, 0);
    // a cluster (along z) takes 16 rows; its warps share the steps of all items
    const int parts = gridDim.z, worker = blockIdx.z * kDownWarps + warp;
    for (int i = lane; i < kTokens * 17; i += 32) acc[warp][0][i] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    const MoeTable& it = *a.table;
    const int nblk = a.inter >> 5, steps = (nblk + 3) >> 2, row0 = blockIdx.x * 16;
    const int64_t pitch = row_bytes(a.inter);
    const int total = it.count * steps;
    const int f0 = (int)((int64_t)total * worker / (parts * kDownWarps)),
              f1 = (int)((int64_t)total * (worker + 1) / (parts * kDownWarps));
    __syncthreads();  // the zeros
    const bool words = !(nblk & 3);
    uint8_t* const own = ring + warp * (RING * S::kBytes);
    const uint32_t base = smem_u32(own);
    const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(zero);
    int li = f0 / steps, ls = f0 - li * steps, lf = f0, lpairs = 0;  // what is copied next
    uint32_t lslot = base;
    TilePtr lp;
    const char* lx[NP];
    const float* le;  // factors of token `lane` of the item
    auto aim = [&] {
        if (lf >= f1) return;
        lp = tile_at<BITS>(a.down, (int64_t)it.expert[li] * a.hidden + row0, ls, nblk);
        const int n = it.n[li];
        lpairs = (n + 1) >> 1;
        auto at = [&](int i) {
            const int row = it.row[li][i];
            return (row & 255) * a.top_k + (row >> 8);
        };
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = 2 * p + (lane >> 4);
            lx[p] = a.h + (i < n ? at(i) : a.tokens * a.top_k) * pitch + ls * 256 + (lane & 15) * 16;
        }
        // (a token that is not there: any factors, its sums are not used)
        le = a.he + ((int64_t)at(lane < n ? lane : 0) * steps + ls) * 4;
    };
    auto issue = [&] {
        if (lf < f1) {
            copy_weights<BITS, NP>(lslot, lp, words, nblk - ls * 4);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                if (p < lpairs) copy16(lslot + S::kInputs + p * 512 + lane * 16, lx[p], true);
                lx[p] += 256;
            }
            if (lane < 2 * lpairs) copy16(lslot + S::kFactors + lane * 16, le, true);
            le += 4;
            ++lf;
            if (++ls == steps) {
                ls = 0;
                ++li;
                aim();
            }
        }
        copies_end();
        lslot = lslot == base + (RING - 1) * S::kBytes ? base : lslot + S::kBytes;
    };
    aim();
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) issue();
    int item = f0 / steps, step = f0 - item * steps, n = 0, pairs = 0;
    float y[NP][2];
    auto begin = [&] {
        n = it.n[item];
        pairs = (n + 1) >> 1;
#pragma unroll
        for (int p = 0; p < NP; ++p) y[p][0] = y[p][1] = 0.f;
    };
    auto finish = [&] {
        __syncwarp();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (p >= pairs) break;
            const float v0 = y[p][0] + __shfl_xor_sync(0xffffffffu, y[p][0], 1);
            const float v1 = y[p][1] + __shfl_xor_sync(0xffffffffu, y[p][1], 1);
            const int k = 2 * p + ((lane & 3) >> 1);
            if (!(lane & 1) && k < n) {
                const int t = it.row[item][k] & 255;
                acc[warp][t][lane >> 2] += v0;
                acc[warp][t][(lane >> 2) + 8] += v1;
            }
        }
    };
    if (f0 < f1) begin();
    const uint8_t* slot = own;
    for (int f = f0; f < f1; ++f) {
        copies_wait<RING - 2>();
        __syncwarp();  // everyone's copies are there, and the slot before is read
        issue();
        do_step<BITS, NP, true>(slot, zeros, a.down.z != nullptr, pairs, y);
        slot = slot == own + (RING - 1) * S::kBytes ? own : slot + S::kBytes;
        if (++step == steps) {
            finish();
            step = 0;
            ++item;
            if (f + 1 < f1) begin();
        }
    }
    if (f0 < f1 && step != 0) finish();
    __syncthreads();
    // the warps' sums in order, then the CTAs'
    for (int i = tid; i < a.tokens * 16; i += kDownWarps * 32) {
        const int t = i >> 4, r = i & 15;
        float v = acc[0][t][r];
#pragma unroll
        for (int w = 1; w < kDownWarps; ++w) v += acc[w][t][r];
        acc[0][t][r] = v;
        if (parts == 1) a.y[(int64_t)t * a.hidden + row0 + r] = __float2half_rn(v);
    }
    if (parts > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (blockIdx.z == 0) {
            for (int i = tid; i < a.tokens * 16; i += kDownWarps * 32) {
                const int t = i >> 4, r = i & 15;
                float v = acc[0][t][r];
                for (int c = 1; c < parts; ++c) v += ld_peer_f32(smem_u32(&acc[0][t][r]), c);
                a.y[(int64_t)t * a.hidden + row0 + r] = __float2half_rn(v);
            }
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Offsets of the workspace's parts, 256-byte aligned.
struct MoeLayout {
    int64_t table, xs, h, he, bytes;
};

MoeLayout moe_layout(const mnb_moe_layer* l, int64_t M) {
    auto up = [](int64_t n) { return (n + 255) & ~(int64_t)255; };
    MoeLayout o;
    o.table = up(M * l->experts * 8);
    o.xs = o.table + up(sizeof(MoeTable));
    o.h = o.xs + (M + 1) * row_bytes(l->hidden);
    o.he = o.h + (M * l->top_k + 1) * row_bytes(l->inter);
    o.bytes = o.he + up(M * l->top_k * (row_bytes(l->inter) / 64) * 4);
    return o;
}

int moe_check(const mnb_moe_layer* l, int64_t M) {
    if (!l || M < 0 || l->hidden <= 0 || l->inter <= 0 || l->experts <= 0 || l->top_k <= 0 || l->top_k > l->experts ||
        (l->flags & ~MNB_MOE_NORMALIZE))
        return MNB_ERR_ARG;
    if ((l->bits != 4 && l->bits != 8) || l->hidden % 32 || l->inter % 32 || l->hidden > 32768 || l->inter > 65536 ||
        l->experts > kMaxExperts || l->top_k > kMaxTop || M > kTokens)
        return MNB_ERR_UNSUPPORTED;
    return MNB_OK;
}

// Dynamic shared memory of the rings; above 48 KB a kernel has to be allowed it (moe_prepare).
template <int BITS, int NP, int WARPS, int RING>
constexpr size_t kRingBytes = (size_t)WARPS * RING * Slot<BITS, NP>::kBytes;

// The up kernel's grid: as many CTAs as run at once, or as there can be units.
template <int BITS, int NP, int SLICES, int RING, int CTAS>
cudaError_t up_launch(const MoeArgs* a, int64_t units, int sms, cudaStream_t st) {
    constexpr size_t smem = kRingBytes<BITS, NP, SLICES * 4, RING>;
    const auto kernel = moe_up_kernel<BITS, NP, SLICES, RING, CTAS>;
    if (!a) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    const int64_t slots = (int64_t)CTAS * sms;
    return launch_pdl(kernel, dim3((unsigned)(units < slots ? units : slots)), dim3(SLICES * 128), smem, st, *a);
}

template <int BITS, int NP, int RING, int CTAS>
cudaError_t down_launch(const MoeArgs* a, int sms, cudaStream_t st) {
    constexpr size_t smem = kRingBytes<BITS, NP, kDownWarps, RING>;
    const auto kernel = moe_down_kernel<BITS, NP, RING, CTAS>;
    if (!a) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    const int tiles = a->hidden / 16;
    int parts = CTAS * sms / tiles;  // CTAs of 16 rows: as many as fit, at most eight
    parts = parts < 1 ? 1 : parts > 8 ? 8 : parts;
    return launch_pdl(kernel, dim3(tiles, 1, parts), dim3(kDownWarps * 32), smem, st, *a, parts);
}

// The two kernels for items of `item` tokens; without arguments, what has to be set up for them.
template <int BITS>
cudaError_t moe_kernels(const MoeArgs* a, int item, bool few, int64_t units, int sms, cudaStream_t st) {
    cudaError_t e;
    if (item == 2) {
        // few units: four warps share a row's inputs, so that there are loads enough on their way
        e = few ? up_launch<BITS, 1, 4, 3, BITS == 4 ? 2 : 1>(a, units, sms, st)
                : up_launch<BITS, 1, 2, BITS == 4 ? 4 : 3, BITS == 4 ? 3 : 2>(a, units, sms, st);
        return e != cudaSuccess ? e : down_launch<BITS, 1, 4, BITS == 4 ? 6 : 4>(a, sms, st);
    }
    if (item == 4) {
        e = up_launch<BITS, 2, 2, 3, BITS == 4 ? 3 : 2>(a, units, sms, st);
        return e != cudaSuccess ? e : down_launch<BITS, 2, 3, BITS == 4 ? 6 : 4>(a, sms, st);
    }
    e = up_launch<BITS, 4, 2, 3, BITS == 4 ? 2 : 1>(a, units, sms, st);
    return e != cudaSuccess ? e : down_launch<BITS, 4, 3, BITS == 4 ? 4 : 3>(a, sms, st);
}

cudaError_t moe_launch(MoeArgs& a, int sms, cudaStream_t st) {
    const cudaError_t e = launch_pdl(moe_router_kernel, dim3(a.experts + 1, (a.tokens + kRouterTokens - 1) / kRouterTokens),
                                     dim3(kRouterThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    // tokens of an item: two where there are no more; four where an expert gets two on average, since more cost
    // registers and a rare expert of many is read again from the cache; else eight
    const int picks = a.tokens * a.top_k;
    a.item = a.tokens <= 2 ? 2 : picks <= 2 * a.experts ? 4 : 8;
    const int64_t units = (int64_t)picks * (a.inter / kTile);
    const bool few = units <= 2 * (int64_t)sms;
    return a.bits == 4 ? moe_kernels<4>(&a, a.item, few, units, sms, st) : moe_kernels<8>(&a, a.item, few, units, sms, st);
}

}  // namespace

cudaError_t moe_prepare() {
    for (int item = 2; item <= 8; item *= 2)
        for (int few = 0; few <= (item == 2); ++few) {
            cudaError_t e = moe_kernels<4>(nullptr, item, few != 0, 0, 0, nullptr);
            if (e == cudaSuccess) e = moe_kernels<8>(nullptr, item, few != 0, 0, 0, nullptr);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

}  // namespace mnb

extern "C" int64_t mnb_moe_workspace(const mnb_moe_layer* layer, int64_t M) {
    const int rc = mnb::moe_check(layer, M);
    return rc != MNB_OK ? rc : mnb::moe_layout(layer, M).bytes;
}

extern "C" int mnb_moe(const mnb_moe_layer* layer, const void* X, int64_t M, void* Y, int32_t* ids, float* weights,
                       void* ws, int64_t ws_bytes, void* stream) {
    using namespace mnb;
    int rc = moe_check(layer, M);
    if (rc != MNB_OK) return rc;
    if (M == 0) return MNB_OK;
    const mnb_moe_layer& l = *layer;
    const MoeLayout o = moe_layout(layer, M);
    if (!X || !Y || X == Y || !l.router || !l.up_Wq || !l.up_scales || !l.down_Wq || !l.down_scales || !ws ||
        ws_bytes < o.bytes)
        return MNB_ERR_ARG;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(l.router, 16) || !aligned(l.up_Wq, 16) ||
        !aligned(l.up_scales, 16) || !aligned(l.down_Wq, 16) || !aligned(l.down_scales, 16) || !aligned(l.up_zp, 4) ||
        !aligned(l.down_zp, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(ws, 16))
        return MNB_ERR_ALIGN;
    int sms;
    unsigned int* status;
    rc = device_ready(&sms, &status);
    if (rc != MNB_OK) return rc;
    char* w = static_cast<char*>(ws);
    MoeArgs a = {};
    a.hidden = l.hidden;
    a.inter = l.inter;
    a.experts = l.experts;
    a.top_k = l.top_k;
    a.tokens = (int)M;
    a.normalize = l.flags & MNB_MOE_NORMALIZE;
    a.bits = l.bits;
    a.x = static_cast<const __half*>(X);
    a.router = static_cast<const __half*>(l.router);
    a.up = {static_cast<const uint8_t*>(l.up_Wq), static_cast<const __half*>(l.up_scales),
            static_cast<const uint8_t*>(l.up_zp)};
    a.down = {static_cast<const uint8_t*>(l.down_Wq), static_cast<const __half*>(l.down_scales),
              static_cast<const uint8_t*>(l.down_zp)};
    a.logits = reinterpret_cast<double*>(w);
    a.table = reinterpret_cast<MoeTable*>(w + o.table);
    a.xs = w + o.xs;
    a.h = w + o.h;
    a.he = reinterpret_cast<float*>(w + o.he);
    a.y = static_cast<__half*>(Y);
    a.ids = ids;
    a.weights = weights;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return moe_launch(a, sms, st) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
