// moe.cu -- a mixture-of-experts layer of block-quantized gated MLPs for up to 16 tokens
// (mnb_moe): three kernels, each started before the one ahead of it ends.
//
//   router   logits x . r_e, one CTA an expert and four tokens.  Which expert comes first decides the
//            output, so the sums are held in two FP32 words each (products of FP16 are exact).
//   up       every CTA picks the experts again from the logits (a warp a token), makes the
//            list of (expert, up to 8 of its tokens) and takes units of 32 features of one
//            item: gate and up rows, eight warps of 16 rows by half of the inputs.
//   down     a CTA takes 16 outputs over all items, so the sum over experts stays in it.
//
// The weights are streamed from memory into registers, 16 bytes a lane: a quad's lanes hold
// four neighbouring blocks of 32 inputs of a row.  A lane takes the zero point of its own
// block off (exact in FP16) and the rows go to the MMA (m16n8k16) as its left operand.
// A step's columns are two tokens by the quad's four blocks: the right operand is zero
// but where a column's block is the lane's own, so each column sums one block of one
// token, exact codes times FP16 inputs in FP32, and the block's scale multiplies its sum in FP32.
// No code is rounded and no sum over K is needed for the zero points.  Two tokens a
// step use a quarter of the MMA's work; an expert of a few tokens' step has one or two.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_batch.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kTokens = MNB_MOE_MAX_TOKENS;
constexpr int kMaxExperts = 256;
constexpr int kMaxTop = 16;
constexpr int kItem = 8;                   // tokens of an item
constexpr int kPairs = kItem / 2;
constexpr int kMaxItems = kTokens * kMaxTop;
// steps (of four blocks) that a warp's loads run ahead: as many as the registers hold
template <int BITS> constexpr int kAhead = BITS == 4 ? 4 : 2;
constexpr int kUpWarps = 8;
constexpr int kTile = 32;                  // features of a unit of the up kernel

struct MoeWeight {
    const uint8_t* q;
    const __half* s;
    const uint8_t* z;
};

struct MoeArgs {
    int hidden, inter, experts, top_k, tokens, normalize;
    const __half* x;
    const __half* router;
    MoeWeight up, down;
    double* logits;       // [tokens, experts]
    int32_t* sel;         // [tokens, top_k]
    __half* h;            // [tokens * top_k, inter]: silu(gate) up / 2^e, e of each 32
    float* he;            // [tokens * top_k, inter / 32]: weight * 2^e
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

__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a) {
    __shared__ double part[kRouterThreads / 32][kRouterTokens];
    const int tid = threadIdx.x, lane = tid & 31, e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
    pdl_wait();
    pdl_launch_dependents();
    const int n = min(a.tokens - t0, kRouterTokens), pieces = a.hidden >> 3;
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
    int count;
    uint16_t expert[kMaxItems];
    uint8_t n[kMaxItems];                  // tokens of the item
    uint16_t row[kMaxItems][kItem];        // token | slot << 8
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
        for (int i = 1; i < kEach; ++i)
            if (key[i] > best) best = key[i], bv = v[i], be = i * 32 + lane;
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
        for (int i = 0; i < kEach; ++i)
            if (e == i * 32 + lane) key[i] = 0;
    }
    float w = lane < a.top_k ? exp_of(mine - top) : 0.f, sum = 0.f;
    if (a.normalize) {
        sum = w;
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i * 32 + lane < a.experts) sum += exp_of(v[i] - top);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane < a.top_k) weight[lane] = __fdiv_rn(w, sum);
}

// The items of the chosen experts (sel in place): by expert number, eight tokens each. Whole CTA.
__device__ void moe_items(const MoeArgs& a, MoeItems& it) {
    const int tid = threadIdx.x, lane = tid & 31, picks = a.tokens * a.top_k;
    for (int e = tid; e < a.experts; e += blockDim.x) it.mask[e] = 0;
    __syncthreads();
    if (tid < picks) atomicOr(&it.mask[it.sel[tid]], 1u << (tid / a.top_k));
    __syncthreads();
    if (tid < 32) {
        int at = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane, n = e < a.experts ? __popc(it.mask[e]) : 0;
            const unsigned one = __ballot_sync(0xffffffffu, n > 0), two = __ballot_sync(0xffffffffu, n > kItem);
            const unsigned below = (1u << lane) - 1u;
            const int first = at + __popc(one & below) + __popc(two & below);
            if (n > 0) {
                it.first[e] = (uint16_t)first;
                it.expert[first] = (uint16_t)e;
                it.n[first] = (uint8_t)min(n, kItem);
                if (n > kItem) {
                    it.expert[first + 1] = (uint16_t)e;
                    it.n[first + 1] = (uint8_t)(n - kItem);
                }
            }
            at += __popc(one) + __popc(two);
        }
        if (lane == 0) it.count = at;
    }
    __syncthreads();
    if (tid < picks) {
        const int t = tid / a.top_k, e = it.sel[tid];
        const int at = __popc(it.mask[e] & ((1u << t) - 1u));
        it.row[it.first[e] + at / kItem][at % kItem] = (uint16_t)(t | (tid - t * a.top_k) << 8);
    }
    __syncthreads();
}

// ---- 16 rows of weights times an item's tokens -------------------------------

__device__ __forceinline__ uint4 ld_stream(const void* p) {  // read once: no place in L1
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// A lane's block of rows g and g + 8: codes, scales (two FP16) and zero points.
template <int BITS>
struct Raw {
    uint4 a[BITS / 4], b[BITS / 4];
    uint32_t s;
    uint32_t za, zb;
};

// Where a lane's blocks of a row tile lie.
struct TilePtr {
    const uint8_t* q;
    const __half* s;
    const uint8_t* z;
};

template <int BITS>
__device__ __forceinline__ TilePtr tile_at(const MoeWeight& w, int64_t row, int nblk) {
    const int lane = threadIdx.x & 31;
    const int64_t at = (row + (lane >> 2)) * nblk + (lane & 3);
    return {w.q + at * (4 * BITS), w.s + at, w.z ? w.z + at : nullptr};
}

template <int BITS>
__device__ __forceinline__ void load_step(Raw<BITS>& r, const TilePtr& p, int step, int nblk) {
    const bool there = step * 4 + (int)(threadIdx.x & 3) < nblk;
    if (there) {
        const uint8_t* q = p.q + (int64_t)step * (16 * BITS);
        const int64_t eight = (int64_t)nblk * 8;
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) {
            r.a[i] = ld_stream(q + i * 16);
            r.b[i] = ld_stream(q + eight * (4 * BITS) + i * 16);
        }
        const unsigned short* s = reinterpret_cast<const unsigned short*>(p.s) + step * 4;
        r.s = (uint32_t)s[0] | (uint32_t)s[eight] << 16;
        r.za = r.zb = 1u << (BITS - 1);
        if (p.z) {
            r.za = p.z[step * 4];
            r.zb = p.z[step * 4 + eight];
        }
    } else {
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) r.a[i] = r.b[i] = make_uint4(0, 0, 0, 0);
        r.s = 0;
        r.za = r.zb = 0;
    }
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

// Adds one step (four blocks of 16 rows) times up to eight tokens: y[p][0], y[p][1] are rows g and
// g + 8 of token 2 p + (lane & 3) / 2, blocks 2 (lane & 1) and the one behind it.  x[p]: where in xs
// the row begins whose values this lane hands to the MMA (-1: none); e[p]: where in es the factors of the
// token's blocks begin (-1: no token).
template <int BITS, bool FACTORS>
__device__ __forceinline__ void do_step(const Raw<BITS>& r, int step, int nblk, int pairs, const __half* xs,
                                        const int* x, const float* es, const int* e, float (*y)[2]) {
    const int t = threadIdx.x & 3, block = step * 4 + t;
    const bool there = block < nblk;
    const uint32_t ca = kMagic1024x2 | r.za * 0x00010001u, cb = kMagic1024x2 | r.zb * 0x00010001u;
    const uint32_t da = hsub2_rn(kHalf960x2, ca), db = hsub2_rn(kHalf960x2, cb);
    float c[kPairs][4];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) c[p][0] = c[p][1] = c[p][2] = c[p][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t A[4], B[4];
        if (BITS == 4) {
            codes4(word(r.a[0], j), ca, da, A);
            codes4(word(r.b[0], j), cb, db, B);
        } else {
            constexpr int kHi = BITS / 4 - 1;
            codes8(word(r.a[j / 2 * kHi], 2 * j % 4), word(r.a[j / 2 * kHi], (2 * j + 1) % 4), ca, A);
            codes8(word(r.b[j / 2 * kHi], 2 * j % 4), word(r.b[j / 2 * kHi], (2 * j + 1) % 4), cb, B);
        }
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            if (p >= pairs) break;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (x[p] >= 0 && there) v = *reinterpret_cast<const uint4*>(xs + (x[p] + block * 32 + j * 8));
            if (BITS == 4) {  // the codes' order: 0 4, 1 5, 2 6, 3 7
                mma_16816(c[p], A[0], B[0], A[1], B[1], prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u));
                mma_16816(c[p], A[2], B[2], A[3], B[3], prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
            } else {
                mma_16816(c[p], A[0], B[0], A[1], B[1], v.x, v.y);
                mma_16816(c[p], A[2], B[2], A[3], B[3], v.z, v.w);
            }
        }
    }
    // scales of the two blocks that this lane holds sums of
    const int from = (threadIdx.x & 28) | (t & 1) * 2;
    const uint32_t s0 = __shfl_sync(0xffffffffu, r.s, from), s1 = __shfl_sync(0xffffffffu, r.s, from + 1);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&s0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&s1));
    const int first = step * 4 + (t & 1) * 2;
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        if (p >= pairs) break;
        float e0 = 1.f, e1 = 1.f;
        if (FACTORS) {
            e0 = e[p] >= 0 && first < nblk ? es[e[p] + first] : 0.f;
            e1 = e[p] >= 0 && first + 1 < nblk ? es[e[p] + first + 1] : 0.f;
        }
        y[p][0] = fmaf(f1.x * e1, c[p][1], fmaf(f0.x * e0, c[p][0], y[p][0]));
        y[p][1] = fmaf(f1.y * e1, c[p][3], fmaf(f0.y * e0, c[p][2], y[p][1]));
    }
}

// ---- gate and up -------------------------------------------------------------

constexpr int kRedPitch = kItem + 1;

template <int BITS>
__global__ void __launch_bounds__(kUpWarps * 32, 2) moe_up_kernel(const MoeArgs a) {
    __shared__ MoeItems it;
    __shared__ float red[2][2][4][16][kRedPitch];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();
    for (int t = warp; t < a.tokens; t += kUpWarps)
        moe_choose(a, t, it.sel + t * a.top_k, it.weight + t * a.top_k);
    __syncthreads();
    if (blockIdx.x == 0 && tid < a.tokens * a.top_k) {
        a.sel[tid] = it.sel[tid];
        if (a.ids) a.ids[tid] = it.sel[tid];
        if (a.weights) a.weights[tid] = it.weight[tid];
    }
    moe_items(a, it);

    const int nblk = a.hidden >> 5, steps = (nblk + 3) >> 2, tiles = a.inter / kTile;
    const int units = it.count * tiles;
    const int q = warp & 3, slice = warp >> 2;  // gate, gate + 16, up, up + 16; half of the inputs
    const int s0 = slice ? (steps + 1) >> 1 : 0, s1 = slice ? steps : (steps + 1) >> 1;
    const int chunks = (((steps + 1) >> 1) + kAhead<BITS> - 1) / kAhead<BITS>;
    auto tile_of = [&](int u) {
        const int item = u / tiles, tile = u - item * tiles;
        return tile_at<BITS>(a.up, (int64_t)it.expert[item] * 2 * a.inter + (q >> 1) * a.inter + tile * kTile +
                                       (q & 1) * 16, nblk);
    };
    Raw<BITS> raw[kAhead<BITS>];
    int lu = blockIdx.x, lc = 0;  // what is loaded next
    TilePtr lp = {};
    if (lu < units) lp = tile_of(lu);
    auto issue = [&](int i) {
        const int s = s0 + lc * kAhead<BITS> + i;
        if (lu < units && s < s1) load_step<BITS>(raw[i], lp, s, nblk);
    };
    auto advance = [&] {
        if (++lc == chunks) {
            lc = 0;
            lu += gridDim.x;
            if (lu < units) lp = tile_of(lu);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead<BITS>; ++i) issue(i);
    advance();
    int buf = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
        const int item = u / tiles, tile = u - item * tiles, n = it.n[item], pairs = (n + 1) >> 1;
        int x[kPairs];
        float y[kPairs][2];
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const int i = 2 * p + (lane >> 4);  // column g: token g / 4, block g % 4
            x[p] = i < n && ((lane >> 2) & 3) == (lane & 3) ? (it.row[item][i] & 255) * a.hidden : -1;
            y[p][0] = y[p][1] = 0.f;
        }
        for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int i = 0; i < kAhead<BITS>; ++i) {
                const int s = s0 + c * kAhead<BITS> + i;
                if (s < s1) do_step<BITS, false>(raw[i], s, nblk, pairs, a.x, x, nullptr, nullptr, y);
                issue(i);
            }
            advance();
        }
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            if (p >= pairs) break;
            const float v0 = y[p][0] + __shfl_xor_sync(0xffffffffu, y[p][0], 1);
            const float v1 = y[p][1] + __shfl_xor_sync(0xffffffffu, y[p][1], 1);
            if (!(lane & 1)) {
                red[buf][slice][q][lane >> 2][2 * p + ((lane & 3) >> 1)] = v0;
                red[buf][slice][q][(lane >> 2) + 8][2 * p + ((lane & 3) >> 1)] = v1;
            }
        }
        __syncthreads();
        if (warp < n) {  // a warp a token, a lane a feature
            const int f = lane;
            const float gate = red[buf][0][f >> 4][f & 15][warp] + red[buf][1][f >> 4][f & 15][warp];
            const float up = red[buf][0][2 + (f >> 4)][f & 15][warp] + red[buf][1][2 + (f >> 4)][f & 15][warp];
            const float h = gate / (1.f + expf(-gate)) * up;
            float m = fabsf(h);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            // FP16 holds the block about its largest value, whatever that is: 2^e <= m < 2^(e + 1)
            uint32_t e = __float_as_uint(m) & 0x7F800000u;
            e = e == 0 || e >= 0x7F000000u ? 0x3F800000u : e;
            const int row = it.row[item][warp], at = (row & 255) * a.top_k + (row >> 8);
            a.h[(int64_t)at * a.inter + tile * kTile + f] = __float2half_rn(h * __uint_as_float(0x7F000000u - e));
            if (lane == 0) a.he[(int64_t)at * tiles + tile] = it.weight[at] * __uint_as_float(e);
        }
    }
}

// ---- down ----------------------------------------------------------------------

template <int BITS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) moe_down_kernel(const MoeArgs a) {
    __shared__ MoeItems it;
    __shared__ float acc[WARPS][kTokens][17];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = lane; i < kTokens * 17; i += 32) acc[warp][0][i] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    if (tid < a.tokens * a.top_k) it.sel[tid] = a.sel[tid];
    __syncthreads();
    moe_items(a, it);

    const int nblk = a.inter >> 5, steps = (nblk + 3) >> 2, row0 = blockIdx.x * 16;
    const int total = it.count * steps;  // of all items; a warp takes a run of them
    const int f0 = (int)((int64_t)total * warp / WARPS), f1 = (int)((int64_t)total * (warp + 1) / WARPS);
    Raw<BITS> raw[kAhead<BITS>];
    int li = f0 / max(steps, 1), ls = f0 - li * steps, lf = f0;  // what is loaded next
    TilePtr lp = {};
    auto tile_of = [&](int item) {
        return tile_at<BITS>(a.down, (int64_t)it.expert[item] * a.hidden + row0, nblk);
    };
    if (f0 < f1) lp = tile_of(li);
    auto issue = [&](int i) {
        if (lf < f1) {
            load_step<BITS>(raw[i], lp, ls, nblk);
            ++lf;
            if (++ls == steps) {
                ls = 0;
                ++li;
                if (lf < f1) lp = tile_of(li);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead<BITS>; ++i) issue(i);
    int item = f0 / max(steps, 1), step = f0 - item * steps, n = 0, pairs = 0;
    int x[kPairs], e[kPairs];
    float y[kPairs][2];
    auto begin = [&] {
        n = it.n[item];
        pairs = (n + 1) >> 1;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const int i = 2 * p + (lane >> 4), k = 2 * p + ((lane & 3) >> 1);
            const int ri = it.row[item][i], rk = it.row[item][k];
            x[p] = i < n && ((lane >> 2) & 3) == (lane & 3)
                       ? ((ri & 255) * a.top_k + (ri >> 8)) * a.inter : -1;
            e[p] = k < n ? ((rk & 255) * a.top_k + (rk >> 8)) * nblk : -1;
            y[p][0] = y[p][1] = 0.f;
        }
    };
    auto finish = [&] {
        __syncwarp();
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
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
    for (int f = f0; f < f1; f += kAhead<BITS>) {
#pragma unroll
        for (int i = 0; i < kAhead<BITS>; ++i) {
            if (f + i < f1) {
                do_step<BITS, true>(raw[i], step, nblk, pairs, a.h, x, a.he, e, y);
                if (++step == steps) {
                    finish();
                    step = 0;
                    ++item;
                    if (f + i + 1 < f1) begin();
                }
            }
            issue(i);
        }
    }
    if (f0 < f1 && step != 0) finish();
    __syncthreads();
    for (int i = tid; i < a.tokens * 16; i += WARPS * 32) {
        const int t = i >> 4, r = i & 15;
        float v = acc[0][t][r];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) v += acc[w][t][r];
        a.y[(int64_t)t * a.hidden + row0 + r] = __float2half_rn(v);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Offsets of the workspace's parts, 256-byte aligned.
struct MoeLayout {
    int64_t sel, h, he, bytes;
};

MoeLayout moe_layout(const mnb_moe_layer* l, int64_t M) {
    auto up = [](int64_t n) { return (n + 255) & ~(int64_t)255; };
    MoeLayout o;
    o.sel = up(M * l->experts * 8);
    o.h = o.sel + up(M * l->top_k * 4);
    o.he = o.h + up(M * l->top_k * l->inter * 2);
    o.bytes = o.he + up(M * l->top_k * (l->inter / 32) * 4);
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

template <int BITS>
cudaError_t moe_launch(const MoeArgs& a, int sms, cudaStream_t st) {
    cudaError_t e = launch_pdl(moe_router_kernel, dim3(a.experts, (a.tokens + kRouterTokens - 1) / kRouterTokens),
                               dim3(kRouterThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    // at most this many items, of which as many as fit run at once
    const int64_t items = (int64_t)a.tokens * a.top_k, units = items * (a.inter / kTile);
    const int64_t slots = 2 * (int64_t)sms;
    e = launch_pdl(moe_up_kernel<BITS>, dim3((unsigned)(units < slots ? units : slots)), dim3(kUpWarps * 32), 0, st, a);
    if (e != cudaSuccess) return e;
    const int tiles = a.hidden / 16;
    if (tiles <= sms) return launch_pdl(moe_down_kernel<BITS, 16>, dim3(tiles), dim3(512), 0, st, a);
    return launch_pdl(moe_down_kernel<BITS, 8>, dim3(tiles), dim3(256), 0, st, a);
}

}  // namespace

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
    a.x = static_cast<const __half*>(X);
    a.router = static_cast<const __half*>(l.router);
    a.up = {static_cast<const uint8_t*>(l.up_Wq), static_cast<const __half*>(l.up_scales),
            static_cast<const uint8_t*>(l.up_zp)};
    a.down = {static_cast<const uint8_t*>(l.down_Wq), static_cast<const __half*>(l.down_scales),
              static_cast<const uint8_t*>(l.down_zp)};
    a.logits = reinterpret_cast<double*>(w);
    a.sel = reinterpret_cast<int32_t*>(w + o.sel);
    a.h = reinterpret_cast<__half*>(w + o.h);
    a.he = reinterpret_cast<float*>(w + o.he);
    a.y = static_cast<__half*>(Y);
    a.ids = ids;
    a.weights = weights;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = l.bits == 4 ? moe_launch<4>(a, sms, st) : moe_launch<8>(a, sms, st);
    return e == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
