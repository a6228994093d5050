// attn.cu -- causal attention over the 8-bit key/value cache (mnb_attn).
//
// Per query row, with codes k_jd, v_jd (exact integers after subtracting 128)
// and one scale a block of 16 tokens:
//     s_j = scale * ks_b * sum_d q_d k_jd,     o = sum_j e^(s_j - m) vs_b v_j / sum_j e^(s_j - m)
// in one pass over the keys with a running reference.
//
//  * The value scale goes into the exponent: w_j = s_j log2(e) + log2(vs_b), and
//    the reference m is a row's maximum of w as of the last time that mattered: it moves
//    when a lane's part of 32 keys (of 128 in the prompt kernel a row's) sums up to more than
//    2^15.  The second product's operand is then 2^(w_j - m) <= 2^15 whatever the value scales
//    are, and rounded to FP16: 2^-11 of each term, and for terms more than 2^14 below the reference,
//    which are subnormal, 2^-25 of it.  The denominator takes each block's sum times 1 / vs_b,
//    in binary32.
//  * Both products take the codes exactly, with binary32 accumulation (mma.sync
//    m16n8k16).  The first one's are fed as FP16 subnormals q 2^-24 (one byte permute for
//    two codes), the offset 128 sum_d q_d taken off the accumulator before it starts;
//    the second one's, whose sum runs over all keys, as the integers q - 128 themselves
//    (1024 + q less 1152), so that nothing has to cancel at the end.
//  * Keys and values are the LEFT operands (16 keys, 16 values of d), the query rows the
//    columns: consecutive (token, head of the kv head's group) pairs, 8 or 16 of them, so
//    the heads that share a kv head share its bytes, and a decode step of up to
//    eight heads a kv head wastes no half of an MMA.  The probabilities pass from the first
//    product's result to the second one's operand with one 8 x 8 transpose a register.
//
// attn_split_kernel: a CTA of four warps takes one row tile, one kv head and
// `chunk` keys.  Each warp walks its own stages of 32 keys (8 KB of codes at head_dim
// 128) through a ring of cp.async copies of its own, so nothing in the loop
// waits on another warp; the warps' results are joined once at the end, and the
// chunks' by attn_join_kernel where a row tile has more than one, or in the cluster that
// the chunks of a tile form where they are few.  The codes are
// stored with their 16-byte chunks permuted by the row, so that both products'
// operand reads are free of bank conflicts.
//
// Bound by memory, head_dim + 4 / 16 bytes a key, twice: one sequence of 131,071 keys and 8 kv heads
// of 128 takes 49.5 us, 5.4 TB/s.  64 uneven sequences of up to 8,192 take 65 us, 5.0 TB/s: at
// their end few CTAs have work left.  (Chunks of equal work over all sequences ended
// together and took 67: each CTA has more to look up and to join.)  Short calls wait for
// their loads one behind the other (lengths, page, scales and codes, then the join): 577 keys
// of 3 heads of 64 take 4.6 us behind another call.
#include "attn_common.cuh"

namespace mnb {

namespace {

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 3;
constexpr int kMaxCluster = 8;
constexpr int kJoinOneWarp = 8;     // chunks that one warp joins
constexpr int kSplitMostRows = 48;  // of a sequence
constexpr double kSplitMostBytes = 30e6;  // of the keys and values that its tiles read
constexpr int kLongPart = 3072;     // keys
constexpr int kShortChunk = 512;    // keys
constexpr int kLongWalk = 1536;     // keys
__host__ __device__ constexpr int ring_stages(int D) { return D == 64 ? 4 : 2; }  // stages of 32 keys in a warp's ring
constexpr float kCodeUnit = 5.9604644775390625e-8f;           // 2^-24, FP16's smallest subnormal
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

// An 8 x 8 matrix of FP16 values (row g in lanes 4 g .. 4 g + 3, two columns a lane), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_peer_f32x4(uint32_t local_addr, uint32_t rank) {
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote));
    return v;
}

// Byte offset of 16-byte chunk c of row r in a block of 16 rows of D codes.
template <int D>
__device__ __forceinline__ uint32_t block_off(int r, int c) {
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) attn_split_kernel(const AttnArgs a) {
    constexpr int KS = D / 16;               // k-steps of the first product
    constexpr int MT = D / 16;               // row tiles (values' d) of the second
    constexpr int kRows = 8 * NT;
    constexpr int kBlockBytes = kKvBlock * D;
    constexpr int kStageBytes = 4 * kBlockBytes;    // two blocks' keys, then their values
    constexpr int kStages = ring_stages(D);
    constexpr int kCopies = kBlockBytes / 16 / 32;  // 16-byte copies a lane and block, keys or values
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    pdl_wait();
    pdl_launch_dependents();

    const int unit = (int)(blockIdx.x / (unsigned)a.b.kv_heads), head = (int)(blockIdx.x % (unsigned)a.b.kv_heads);
    const int split = a.by_length ? a.splits - 1 - (int)blockIdx.z : (int)blockIdx.z;
    Tile tl;
    if (!find_tile(a, a.by_length ? kv_by_length(a.b, unit) : unit, NT == 1 ? 3 : 4, tl)) return;
    if ((int64_t)tl.n * a.group > a.most_rows) return;  // the prompt kernel's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int rows = (int)min((int64_t)tl.n * a.group - tl.r0, (int64_t)kRows);
    const int first = tl.len - tl.n;  // position of the call's first token

    // the tile: its last token sees furthest, its first one starts furthest back
    const int tok_a = tl.r0 / a.group, tok_b = (tl.r0 + rows - 1) / a.group;
    const int hi_t = min(max(first + tok_b + 1, 0), a.b.max_tokens);  // past the table are no keys
    const int lo_t = window_start(a, first + tok_a);
    const int64_t begin64 = (int64_t)(lo_t & ~(kKvBlock - 1)) + (int64_t)split * a.chunk;
    const int begin = (int)min(begin64, (int64_t)hi_t);
    // the last chunk takes what is left, however long
    const int end = split == a.splits - 1 ? hi_t : (int)min(begin64 + a.chunk, (int64_t)hi_t);
    const int nstage = (end - begin + 2 * kKvBlock - 1) / (2 * kKvBlock);
    const int mine = nstage > warp ? (nstage - warp + kWarps - 1) / kWarps : 0;
    // blocks that every row of the tile sees wholly need no mask
    const int all_hi = min(max(first + tok_a + 1, 0), end);
    const int all_lo = window_start(a, first + tok_b);

    // Where this warp's blocks lie, 32 blocks (16 stages) at a time, one a lane: the row
    // of the cache (-1: no such page) and the two scales; `nxt` is loaded while `cur` is used.
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * kStageBytes);
    const int pmask = (1 << a.b.page_shift) - 1;
    auto stage_pos = [&](int i) { return begin + (warp + i * kWarps) * (2 * kKvBlock); };
    auto lane_pos = [&](int base) { return stage_pos(base + (lane >> 1)) + (lane & 1) * kKvBlock; };
    auto load_page = [&](int base) {
        return base + (lane >> 1) < mine && lane_pos(base) < end ? kv_page(a.b, tl.s, lane_pos(base)) : -1;
    };
    auto slot_of = [&](int page, int base) {
        return page < 0 ? (int64_t)-1
                        : (((int64_t)page * a.b.kv_heads + head) << a.b.page_shift) + (lane_pos(base) & pmask);
    };
    // An infinite key scale becomes NaN: its codes stand for no number, but the scores they give
    // here are zero to a few roundings of either sign, which would make the key count as hidden.
    auto load_scales = [&](int64_t slot, float& ks, float& vs) {
        ks = slot < 0 ? 0.f : a.Ks[slot >> 4];
        ks = fmaf(0.f, ks, ks);
        vs = slot < 0 ? 1.f : a.Vs[slot >> 4];
    };
    int64_t slot_cur = slot_of(load_page(0), 0), slot_nxt = -1;
    int page_nxt = -1;
    float ks_cur, vs_cur, ks_nxt = 0.f, vs_nxt = 1.f;
    load_scales(slot_cur, ks_cur, vs_cur);
    auto issue = [&](int i, int base) {  // stage i of this warp into its ring; one copy group, maybe empty
        if (i < mine) {
            const uint32_t dst = ring + (uint32_t)((i % kStages) * kStageBytes);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t slot = __shfl_sync(0xffffffffu, i - base < 16 ? slot_cur : slot_nxt, 2 * (i & 15) + k);
                if (slot < 0) continue;
                const uint8_t* ksrc = a.K + slot * D + lane * 16;
                const uint8_t* vsrc = a.V + slot * D + lane * 16;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    const int id = lane + 32 * c;
                    const uint32_t off = (uint32_t)(k * kBlockBytes) + block_off<D>(id / (D / 16), id % (D / 16));
                    cp_async16(dst + off, ksrc + 512 * c);
                    cp_async16(dst + 2 * kBlockBytes + off, vsrc + 512 * c);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, 0);

    // Queries as the first product's right operand (column g of tile nt), and the constant
    // each column starts from: codes enter as q 2^-24, so -128 sum_d q_d 2^-24.
    uint32_t qf[NT][KS][2];
    float q0[NT][2];
    int hi[NT][2], lo[NT][2];  // what rows 8 nt + 2 t, + 1 see: [lo, hi)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = tl.r0 + 8 * nt + g, tok = r / a.group;
        const int64_t row = tl.row0 + tok;
        const bool ok = 8 * nt + g < rows && row >= 0 && row < a.b.tokens && mine > 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.Q + (ok ? row * a.q_stride + (int64_t)(head * a.group + (r - tok * a.group)) * D : 0) + t * (D / 4));
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            const uint4 v = ok ? src[j] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qf[nt][2 * j + (i >> 1)][i & 1] = w[i];
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                sum += f.x + f.y;
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            q0[nt][b] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + b)) * (-128.f * kCodeUnit);
            const int rr = 8 * nt + 2 * t + b;
            const int pos = first + (tl.r0 + rr) / a.group;
            hi[nt][b] = rr < rows ? min(max(pos + 1, 0), end) : 0;
            lo[nt][b] = window_start(a, pos);
        }
    }

    float o[MT][NT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][nt][c] = 0.f;
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // columns without a row: a reference that always holds
            m[nt][b] = 8 * nt + 2 * t + b < rows ? -INFINITY : 0.f;
            l[nt][b] = 0.f;
        }

    for (int i = 0; i < mine; ++i) {
        const int base = i & ~15;
        if ((i & 15) == 0) {
            if (i > 0) {
                slot_cur = slot_nxt;
                ks_cur = ks_nxt;
                vs_cur = vs_nxt;
            }
            page_nxt = load_page(base + 16);
        } else if ((i & 15) == 4) {  // the pages have arrived long since
            slot_nxt = slot_of(page_nxt, base + 16);
            load_scales(slot_nxt, ks_nxt, vs_nxt);
        }
        issue(i + kStages - 1, base);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint32_t kb = ring + (uint32_t)((i % kStages) * kStageBytes), vb = kb + 2 * kBlockBytes;

        float sc[2][NT][4], ivs[2];
        bool here[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int from = 2 * (i & 15) + k;
            const float ks = __shfl_sync(0xffffffffu, ks_cur, from) * (a.scale_log2 * (1.f / kCodeUnit));
            const float vs0 = __shfl_sync(0xffffffffu, vs_cur, from);
            here[k] = __shfl_sync(0xffffffffu, slot_cur >= 0 ? 1 : 0, from) != 0;
            // A scale of zero has codes of zero value only: any scale gives the same products.
            // 2^-60 lies below every other scale (2^-31), so it never lifts the maximum.
            const float vs = vs0 == 0.f ? 8.67361738e-19f : vs0;
            const float lv = __log2f(vs);
            ivs[k] = __frcp_rn(vs);
            // S^T = K Q^T: rows g, g + 8 are keys, columns 2t, 2t + 1 query rows
            uint32_t w[2][KS];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 v =
                        lds128(kb + (uint32_t)(k * kBlockBytes) + block_off<D>(g + 8 * h, t * (D / 64) + c));
                    w[h][4 * c] = v.x;
                    w[h][4 * c + 1] = v.y;
                    w[h][4 * c + 2] = v.z;
                    w[h][4 * c + 3] = v.w;
                }
            float odd[NT][4];  // a second accumulator: half the way through dependent products
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[k][nt][0] = sc[k][nt][2] = q0[nt][0];
                sc[k][nt][1] = sc[k][nt][3] = q0[nt][1];
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t a0 = prmt(w[0][j], 0u, 0x4140u), a1 = prmt(w[1][j], 0u, 0x4140u);
                const uint32_t a2 = prmt(w[0][j], 0u, 0x4342u), a3 = prmt(w[1][j], 0u, 0x4342u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (j == 1)
                        mma_16816_z(odd[nt], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
                    else
                        mma_16816(j & 1 ? odd[nt] : sc[k][nt], a0, a1, a2, a3, qf[nt][j][0], qf[nt][j][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) sc[k][nt][c] = fmaf(sc[k][nt][c] + odd[nt][c], ks, lv);
        }
        const int p0 = stage_pos(i);
        if (!here[0] || !here[1] || p0 < all_lo || p0 + 2 * kKvBlock > all_hi) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = p0 + 16 * k + g + 8 * (c >> 1), b = c & 1;
                        if (!here[k] || j >= hi[nt][b] || j < lo[nt][b]) sc[k][nt][c] = -INFINITY;
                    }
        }
        // The reference m holds for most stages: FP16 takes probabilities up to 2^15 about it as
        // exactly as up to 1, and a lane's sum says so.  Else the warp goes through the maximum.
        float pr[2][NT][4];
        float sum[2][NT][2];
        auto probabilities = [&]() {
            bool holds = true;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float mu = m[nt][b] == -INFINITY ? 0.f : m[nt][b];  // a row that has seen nothing yet
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pr[k][nt][b] = ex2(sc[k][nt][b] - mu);
                        pr[k][nt][b + 2] = ex2(sc[k][nt][b + 2] - mu);
                        sum[k][nt][b] = pr[k][nt][b] + pr[k][nt][b + 2];
                    }
                    holds = holds && m[nt][b] != -INFINITY && sum[0][nt][b] + sum[1][nt][b] <= 32768.f;
                }
            return holds;
        };
        if (!__all_sync(0xffffffffu, probabilities())) {
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float x = fmaxf(fmaxf(sc[0][nt][b], sc[0][nt][b + 2]), fmaxf(sc[1][nt][b], sc[1][nt][b + 2]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    x = fmaxf(x, m[nt][b]);
                    f[nt][b] = ex2(m[nt][b] - (x == -INFINITY ? 0.f : x));
                    m[nt][b] = x;
                    l[nt][b] *= f[nt][b];
                }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[j][nt][c] *= f[nt][c & 1];
            probabilities();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k)  // a block hidden from the row may have any scale
                    if (sum[k][nt][b] != 0.f) l[nt][b] = fmaf(sum[k][nt][b], ivs[k], l[nt][b]);
        // P^T as the second product's right operand: columns are query rows, k the keys
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                pf[k][nt][0] = transpose8(pack_half2(pr[k][nt][0], pr[k][nt][1]));
                pf[k][nt][1] = transpose8(pack_half2(pr[k][nt][2], pr[k][nt][3]));
            }

        // O^T += V^T P^T: lane (g, t) holds the codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 at
        // d = (D / 8) g + e; row tile j has e = 2j in its row g and 2j + 1 in its row g + 8
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t v[4][D / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 2 * t + (r & 1) + 8 * (r >> 1);
                const uint32_t at = vb + (uint32_t)(k * kBlockBytes);
                if constexpr (D == 128) {
                    const uint4 x = lds128(at + block_off<D>(row, g));
                    v[r][0] = x.x;
                    v[r][1] = x.y;
                    v[r][2] = x.z;
                    v[r][3] = x.w;
                } else {
                    const uint2 x = lds64(at + block_off<D>(row, g >> 1) + (uint32_t)((g & 1) * 8));
                    v[r][0] = x.x;
                    v[r][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the two keys of a pair side by side: bytes (d, d, d + 1, d + 1)
                    const uint32_t x = prmt(v[0][w], v[1][w], h ? 0x7362u : 0x5140u);
                    const uint32_t y = prmt(v[2][w], v[3][w], h ? 0x7362u : 0x5140u);
                    const uint32_t a0 = codes_half2<0x4140u>(x), a1 = codes_half2<0x4342u>(x);
                    const uint32_t a2 = codes_half2<0x4140u>(y), a3 = codes_half2<0x4342u>(y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816(o[2 * w + h][nt], a0, a1, a2, a3, pf[k][nt][0], pf[k][nt][1]);
                }
        }
        __syncwarp();  // the stage is read before it is filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[nt][b] += __shfl_xor_sync(0xffffffffu, l[nt][b], x);
            if (g == 0) {
                s_m[warp][8 * nt + 2 * t + b] = m[nt][b];
                s_l[warp][8 * nt + 2 * t + b] = l[nt][b];
            }
        }
    __syncthreads();  // also: every ring is free
    constexpr int kPitch = D + 4;
    float* s_o = reinterpret_cast<float*>(smem);  // [kWarps][kRows][kPitch]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = 8 * nt + 2 * t + b;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][row]);
            const float fac = ex2(m[nt][b] - (mm == -INFINITY ? 0.f : mm));
            float* dst = s_o + (warp * kRows + row) * kPitch + g * (D / 8);
#pragma unroll
            for (int j = 0; j < MT; j += 2)
                *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[j][nt][b] * fac, o[j][nt][b + 2] * fac,
                                                                      o[j + 1][nt][b] * fac, o[j + 1][nt][b + 2] * fac);
        }
    __syncthreads();
    // kPer threads a row, four values at a time
    constexpr int kPer = kWarps * 32 / kRows;
    const int row = threadIdx.x / kPer, part = threadIdx.x % kPer;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][row]);
    const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ll += s_l[w][row] * ex2(s_m[w][row] - mu);
    const int r = tl.r0 + row, tok = r / a.group;
    const int64_t trow = tl.row0 + tok;
    const bool ok = row < rows && trow >= 0 && trow < a.b.tokens;
    const int qh = head * a.group + (r - tok * a.group);
    const int64_t orow = trow * a.q_heads + qh;
    auto warps_sum = [&](int d) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kRows + row) * kPitch + d);
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
        }
        return sum;
    };
    auto put = [&](int d, float4 x, float inv) {
        *reinterpret_cast<uint2*>(a.out + trow * a.out_stride + (int64_t)qh * D + d) =
            make_uint2(pack_half2(x.x * inv, x.y * inv), pack_half2(x.z * inv, x.w * inv));
    };
    auto put_lse = [&](float ref, float den) {
        if (a.lse) a.lse[orow] = den == 0.f ? -INFINITY : (ref + log2f(den)) * kLn2;
    };
    if (!a.cluster) {
        if (!ok) return;
        const float inv = a.splits > 1 ? 1.f : (ll == 0.f ? 0.f : __fdiv_rn(1.f, ll));
#pragma unroll
        for (int d = part * 4; d < D; d += kPer * 4) {
            const float4 sum = warps_sum(d);
            if (a.splits > 1)
                *reinterpret_cast<float4*>(a.part + (orow * a.splits + split) * D + d) = sum;
            else
                put(d, sum, inv);
        }
        if (part == 0) {
            if (a.splits > 1)
                *reinterpret_cast<float2*>(a.ml + (orow * a.splits + split) * 2) = make_float2(mm, ll);
            else
                put_lse(mu, ll);
        }
        return;
    }
    // Up to eight chunks are one cluster: the CTAs leave their sums in their own shared memory,
    // and each joins every splits-th piece of four values, the chunks in their order.
    float* c_o = s_o + kWarps * kRows * kPitch;  // [kRows][D]
    float* c_m = c_o + kRows * D;                // [kRows][2]
#pragma unroll
    for (int d = part * 4; d < D; d += kPer * 4) *reinterpret_cast<float4*>(c_o + row * D + d) = warps_sum(d);
    if (part == 0) {
        c_m[2 * row] = mm;
        c_m[2 * row + 1] = ll;
    }
    cluster_sync();
    if (ok) {
        const uint32_t m_at = smem_u32(c_m + 2 * row), o_at = smem_u32(c_o + row * D);
        float cm[kMaxCluster], cl[kMaxCluster], ref = -INFINITY, den = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            cm[c] = c < a.splits ? ld_peer_f32(m_at, (uint32_t)c) : -INFINITY;
            cl[c] = c < a.splits ? ld_peer_f32(m_at + 4u, (uint32_t)c) : 0.f;
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) ref = fmaxf(ref, cm[c]);
        const float u = ref == -INFINITY ? 0.f : ref;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            cm[c] = ex2(cm[c] - u);
            if (c < a.splits) den = fmaf(cl[c], cm[c], den);
        }
        const float inv = den == 0.f ? 0.f : __fdiv_rn(1.f, den);
        for (int i = split; part + i * kPer < D / 4; i += a.splits) {
            const int d = (part + i * kPer) * 4;
            float4 x[kMaxCluster], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                if (c < a.splits) x[c] = ld_peer_f32x4(o_at + (uint32_t)d * 4u, (uint32_t)c);
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                if (c < a.splits) {
                    sum.x = fmaf(x[c].x, cm[c], sum.x);
                    sum.y = fmaf(x[c].y, cm[c], sum.y);
                    sum.z = fmaf(x[c].z, cm[c], sum.z);
                    sum.w = fmaf(x[c].w, cm[c], sum.w);
                }
            put(d, sum, inv);
        }
        if (part == 0 && split == 0) put_lse(u, den);
    }
    cluster_sync();  // the sums stay until every CTA has read them
}

// The chunks of a row (token, query head) joined: out = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c.
// WARPS warps a row take the chunks in turn, four loads in flight each, and are added in
// their order.  One warp a row while there are few chunks; with more, a row's loads one behind the
// other would be what the call waits for (131,071 keys in 114 chunks: 89 us with one warp a
// row, 53 with eight).
template <int D, int WARPS>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
    constexpr int kRowsPerCta = 8 / WARPS;
    constexpr int V = D / 32;  // values a lane
    __shared__ float s_acc[8][D], s_l[8];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRowsPerCta + warp / WARPS;
    const int w = warp % WARPS;
    const bool ok = row < (int64_t)a.b.tokens * a.q_heads;
    const int splits = ok ? a.splits : 0;
    const float2* ml = reinterpret_cast<const float2*>(a.ml) + row * a.splits;
    float mm = -INFINITY;
    for (int c = lane; c < splits; c += 32) mm = fmaxf(mm, ml[c].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
    const float mu = mm == -INFINITY ? 0.f : mm;
    float acc[V], ll = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    const float* part = a.part + row * a.splits * D + lane * V;
    auto load = [&](int c, float (&v)[V]) {
        if constexpr (V == 4) {
            const float4 p = *reinterpret_cast<const float4*>(part + (int64_t)c * D);
            v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
        } else {
            const float2 p = *reinterpret_cast<const float2*>(part + (int64_t)c * D);
            v[0] = p.x, v[1] = p.y;
        }
    };
    constexpr int kAhead = 4;
    for (int c0 = w; c0 < splits; c0 += WARPS * kAhead) {
        float v[kAhead][V];
        float2 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = min(c0 + i * WARPS, splits - 1);
            load(c, v[i]);
            x[i] = ml[c];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            // a chunk that saw nothing has sums of zero and m = -infinity: factor 0
            const float f = c0 + i * WARPS < splits ? ex2(x[i].x - mu) : 0.f;
            if (c0 + i * WARPS < splits) ll = fmaf(x[i].y, f, ll);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c0 + i * WARPS < splits) acc[j] = fmaf(v[i][j], f, acc[j]);
        }
    }
    if constexpr (WARPS > 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) s_acc[warp][lane * V + j] = acc[j];
        if (lane == 0) s_l[warp] = ll;
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int i = 1; i < WARPS; ++i) {
            ll += s_l[warp + i];
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += s_acc[warp + i][lane * V + j];
        }
    }
    if (!ok) return;
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

constexpr int split_smem(int D, int nt) {
    const int ring = kWarps * ring_stages(D) * 4 * kKvBlock * D;
    const int join = (kWarps * 8 * nt * (D + 4) + 8 * nt * (D + 2)) * 4;  // the warps' sums, the cluster's
    return ring > join ? ring : join;
}

struct AttnPlan {
    int split_rows;      // split kernel: query rows of a tile, 8 or 16; 0: not launched
    int row_tiles;       // prompt kernel: tiles of 128 rows a CTA, 1 or 2; 0: not launched
    int64_t split_units, prompt_units;
    int split_single, prompt_single;  // every sequence of the kernel has at most one tile
    int chunk, splits;   // both kernels'
    int by_length;       // split kernel alone: long sequences first
    int cluster;         // split kernel alone: the CTAs of a row tile are a cluster and join themselves
    int64_t ws_bytes;
};

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Which kernels run, and how the keys are dealt out.  Up to 48 rows (tokens x heads of a kv
// head) a sequence the split kernel is faster, in tiles of 8 or 16 rows that each read the keys
// (35 rows: 13.4 against 17.8 us at 16 x 4,000 keys and 2 kv heads of 64, 20 rows: 110
// against 144 us at 3 x 131,070 and 8 of 128), above it the prompt kernel (64 rows: 153
// against 234 us there), from 129 rows on or where the split kernel's tiles read more than 30 MB (96
// rows, 8 heads of 128: 500 keys 10.3 against 15.3 us, 4,000 keys 16.8 against 14.6).  Where a batch may hold both long prompts and single tokens, the
// sequences of one split tile (8 rows, or 16 with more than 8 heads a kv head) go to the split kernel.
int attn_plan(const mnb_kv_cache* c, const mnb_kv_batch* b, int q_heads, int window, int sms, AttnPlan* p) {
    const int G = q_heads / c->kv_heads, H = c->kv_heads;
    const int64_t most = (int64_t)b->max_new * G;
    // bytes that the split kernel's tiles of 16 rows read (sizes may be absurd: not in integers)
    const double reread = 2.0 * b->seqs * (double)((most + 15) / 16) * H * b->max_len * c->head_dim;
    *p = AttnPlan{};
    const bool prompt = most > kSplitMostRows && (most > kPromptTile || reread > kSplitMostBytes);
    if (!prompt)
        p->split_rows = most <= 8 ? 8 : 16;
    else if (b->seqs > 1 && G <= 16 && b->tokens < (int64_t)b->seqs * b->max_new)
        p->split_rows = G <= 8 ? 8 : 16;
    p->split_single = prompt || most <= p->split_rows;
    p->split_units = p->split_single ? b->seqs : kv_items(b->tokens, b->seqs, {G, p->split_rows == 8 ? 3 : 4, 1});
    // Keys that a tile of so many rows sees at most: all, or with a window its tokens' windows,
    // from a block's start.
    auto keys_of = [&](int rows) {
        int64_t keys = b->max_len > 1 ? b->max_len : 1;
        if (window > 0) keys = min(keys, (int64_t)window + rows / G + 1 + kKvBlock);
        return keys;
    };
    int64_t keys = keys_of(p->split_rows), chunk = 0;
    if (prompt) {
        // One row tile a CTA or two, and keys enough a CTA to fill the SMs, at least 256, 512 or 1024:
        // whichever ends first by this count, in eighths of the time of a step of 128 keys with two
        // tiles (with one it takes 6, a CTA's start and end 22, the join 24): the longest CTA, or
        // all of them over the SMs.  Over 90 sizes (1 to 4 sequences, 40 to 4,096 tokens behind 1 to
        // 8,000, 8 heads of 128 and 2 of 64) what it takes is 1% from the best of them on average, 16%
        // at worst; always two tiles and 512 keys, 11% on average.  600 tokens, 8 heads of 128: 16 us
        // with one tile, 26 with two in two chunks; 4,096 behind 8,000: 895 and 605; 40 behind 1,000: 16
        // and 19.  Several sequences of few tiles and long walks may also get twice the chunks, of
        // which the shorter sequences leave some empty (16 tokens of 4 of up to 30,000 keys: 93 to 58
        // us; with many tiles it costs: 2,000 of 4 behind 8,000, 2 heads of 64: 129 to 146).
        int64_t least = INT64_MAX;
        const int folds = b->seqs > 1 ? 2 : 1;
        for (int i = 0; i < (most <= kPromptTile ? 3 : 6) * folds; ++i) {
            const bool fold = i / 3 % folds == 1;
            const int q = 1 + i / (3 * folds), rows = q * kPromptTile, slots = fold ? 2 * sms : sms;
            const int64_t k = keys_of(rows);
            const bool single = most <= rows;
            const int64_t units = single         ? b->seqs
                                  : b->seqs == 1 ? ((int64_t)b->tokens * G + rows - 1) / rows
                                                 : kv_items(b->tokens, b->seqs, {G, q == 1 ? 7 : 8, 1});
            const int64_t tiles = units * H;
            if (tiles > INT32_MAX) continue;
            int64_t each = tiles >= slots ? k : round_up((tiles * k + slots - 1) / slots, 128);
            each = max(each, (int64_t)(256 << i % 3));
            if (fold && (2 * tiles > sms || each < kLongPart)) continue;
            if (p->split_rows) each = min(each, (int64_t)8192);  // a single token's CTA walks its chunk alone
            auto time = [&](int64_t walk) { return (walk + 127) / 128 * (q == 1 ? 6 : 8) + 22; };
            // causal tiles see fewer and fewer of the new tokens, half of them on average
            const int64_t whole = k / each, rest = k % each, last = max(min(each, k - b->max_new / 2), (int64_t)1);
            int64_t all, cost;
            if (each >= k) {
                all = time(last);
                cost = time(k);
            } else {
                all = (whole - 1) * time(each) + (rest ? time(each) + time(rest) : time(last));
                cost = time(each);
            }
            cost = max(cost, tiles * all * (fold ? 7 : 8) / (8 * (int64_t)sms)) + (each < k ? 24 : 0);
            if (cost >= least) continue;
            least = cost;
            keys = k;
            chunk = each;
            p->row_tiles = q;
            p->prompt_single = single;
            p->prompt_units = units;
        }
    }
    if ((prompt && !p->row_tiles) || p->split_units * H > INT32_MAX) return MNB_ERR_UNSUPPORTED;
    if (!prompt) {
        // Whole rounds of the four warps.  One sequence: a CTA for every slot (131,071 keys: 49.5
        // against 52.7 us with two).  Several, of lengths that are not known here: twice as many, so that
        // the short ones' slots find work (3 uneven ones of up to 131,071 keys: 75 us with
        // one, 59 with two, 67 with three; 64 of up to 8,192: 77, 66 and 64).  But no chunk
        // under 512 keys for that, four stages a warp: what a chunk costs by itself is more
        // then (8 kv heads, 8 sequences of up to 2,000 keys: 9.0 against 10.0 us; 5 tokens of 2 of up to
        // 8,000, 2 kv heads of 64: 9.0 against 13.4), and from there on it is less (32 of 8,000,
        // 8 heads: 35 against 48).
        const int64_t slots = (int64_t)sms * kCtasPerSm, all = p->split_units * H * keys;
        chunk = (all + slots - 1) / slots;
        if (b->seqs > 1 && chunk > kShortChunk) chunk = max((all + 2 * slots - 1) / (2 * slots), (int64_t)kShortChunk);
        chunk = round_up(chunk, kWarps * 2 * kKvBlock);
    }
    if (keys / chunk >= 65535) chunk = round_up(keys / 65535 + 1, 128);
    p->splits = (int)((keys + chunk - 1) / chunk);
    chunk = round_up(chunk, 128);
    p->chunk = (int)(chunk < INT32_MAX - 128 ? chunk : INT32_MAX - 127);
    // Few chunks that all run at once join through shared memory: no second kernel (577 keys of 3
    // heads: 4.6 against 5.8 us).  Not with more CTAs than slots: a cluster waits for its
    // longest chunk, and starts only when there is room for all (64 uneven sequences: 83
    // against 66 us).
    p->cluster = !prompt && p->splits > 1 && p->splits <= kMaxCluster &&
                 p->split_units * H * p->splits <= (int64_t)sms * kCtasPerSm;
    // Of many CTAs the long ones start first, so that the last ones are short: 128 sequences of up to
    // 8,000 keys, 8 kv heads of 128: 96 against 109 us, 256 of them 161 against 189.  Finding the
    // u-th longest costs a CTA half a microsecond: not for short walks (256 of up to 1,000: 41.5
    // against 38.7), nor where few CTAs share a slot (96 of up to 4,000, 2 kv heads of 64: 18.7
    // against 15.8).
    p->by_length = !prompt && p->split_single && b->seqs <= kKvSortMost &&
                   2 * p->split_units * H >= 3 * (int64_t)sms * kCtasPerSm && min(chunk, keys) >= kLongWalk;
    p->ws_bytes = p->splits > 1 && !p->cluster ? (int64_t)b->tokens * q_heads * p->splits * (c->head_dim + 2) * 4 : 0;
    return MNB_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D>
cudaError_t launch(AttnArgs a, const AttnPlan& p, unsigned int* status, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.row_tiles) {
        a.single = p.prompt_single;
        a.skip_rows = p.split_rows;
        e = attn_prompt_launch(a, p.row_tiles, p.prompt_units, status, st);
    }
    if (e == cudaSuccess && p.split_rows) {
        a.single = p.split_single;
        a.most_rows = p.row_tiles ? p.split_rows : INT64_MAX;
        a.by_length = p.by_length;
        const dim3 grid((unsigned)(p.split_units * a.b.kv_heads), 1, (unsigned)p.splits), block(kWarps * 32);
        const int cluster = p.cluster ? p.splits : 1;
        e = p.split_rows == 8 ? launch_pdl(attn_split_kernel<D, 1>, grid, block, split_smem(D, 1), st, a, cluster)
                              : launch_pdl(attn_split_kernel<D, 2>, grid, block, split_smem(D, 2), st, a, cluster);
    }
    if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
    const int64_t rows = (int64_t)a.b.tokens * a.q_heads;
    if (p.splits <= kJoinOneWarp)
        return launch_pdl(attn_join_kernel<D, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a);
    return launch_pdl(attn_join_kernel<D, 8>, dim3((unsigned)rows), dim3(256), 0, st, a);
}

// The checks mnb_attn and mnb_attn_workspace share.
int attn_check(const mnb_kv_cache* c, const mnb_kv_batch* b, int q_heads, int window, bool* empty) {
    const int rc = kv_check(c, b, empty);
    if (rc != MNB_OK) return rc;
    if (q_heads <= 0 || window < 0) return MNB_ERR_ARG;
    if (q_heads % c->kv_heads != 0 || q_heads > 65535) return MNB_ERR_UNSUPPORTED;
    if ((int64_t)b->tokens * q_heads > INT32_MAX) return MNB_ERR_UNSUPPORTED;
    return MNB_OK;
}

// The plan on a GPU of so many SMs (<= 0: the current one); without tokens all zeros.
int attn_plan_for(const mnb_kv_cache* c, const mnb_kv_batch* b, int q_heads, int window, int sms, AttnPlan* p) {
    bool empty;
    int rc = attn_check(c, b, q_heads, window, &empty);
    if (rc != MNB_OK) return rc;
    *p = AttnPlan{};
    if (empty) return MNB_OK;
    unsigned int* status;
    if (sms <= 0 && (rc = device_ready(&sms, &status)) != MNB_OK) return rc;
    return attn_plan(c, b, q_heads, window, sms, p);
}

}  // namespace

cudaError_t attn_prepare() {
    const auto allow = [](const void* f, int bytes) {
        return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    cudaError_t e = allow((const void*)attn_split_kernel<64, 1>, split_smem(64, 1));
    if (e == cudaSuccess) e = allow((const void*)attn_split_kernel<64, 2>, split_smem(64, 2));
    if (e == cudaSuccess) e = allow((const void*)attn_split_kernel<128, 1>, split_smem(128, 1));
    if (e == cudaSuccess) e = allow((const void*)attn_split_kernel<128, 2>, split_smem(128, 2));
    if (e == cudaSuccess) e = attn_prompt_prepare();
    return e;
}

}  // namespace mnb

extern "C" int64_t mnb_attn_workspace(const mnb_kv_cache* cache, const mnb_kv_batch* batch, int32_t q_heads,
                                      int32_t window, int32_t sm_count) {
    mnb::AttnPlan p;
    const int rc = mnb::attn_plan_for(cache, batch, q_heads, window, sm_count, &p);
    return rc != MNB_OK ? rc : p.ws_bytes;
}

extern "C" int mnb_attn_plan(const mnb_kv_cache* cache, const mnb_kv_batch* batch, int32_t q_heads, int32_t window,
                             int32_t sm_count, mnb_attn_plan_info* out) {
    if (!out) return MNB_ERR_ARG;
    mnb::AttnPlan p;
    const int rc = mnb::attn_plan_for(cache, batch, q_heads, window, sm_count, &p);
    if (rc != MNB_OK) return rc;
    *out = {p.row_tiles * mnb::kPromptTile, p.split_rows, p.chunk, p.splits, p.cluster, p.by_length};
    return MNB_OK;
}

extern "C" int mnb_attn(const mnb_kv_cache* cache, const mnb_kv_batch* batch, const void* Q, int64_t q_stride,
                        int32_t q_heads, float scale, int32_t window, void* out, int64_t out_stride, float* lse,
                        void* ws, int64_t ws_bytes, void* stream) {
    bool empty;
    int rc = mnb::attn_check(cache, batch, q_heads, window, &empty);
    if (rc != MNB_OK) return rc;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    // the scale meets key scales and 2^24 in binary32
    if (q_stride < width || out_stride < width || ws_bytes < 0 || !(fabsf(scale) <= 1e27f)) return MNB_ERR_ARG;
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
    a.single = 0;
    a.skip_rows = 0;
    a.most_rows = INT64_MAX;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.cluster = p.cluster;
    a.by_length = 0;
    a.part = static_cast<float*>(ws);
    a.ml = a.part ? a.part + batch->tokens * (int64_t)q_heads * p.splits * cache->head_dim : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->head_dim == 64 ? mnb::launch<64>(a, p, status, st) : mnb::launch<128>(a, p, status, st);
    return e == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}
