// attn_prompt.cu -- attention of many query rows over the 8-bit cache on the
// tensor cores with accumulators in tensor memory (tcgen05), the path of prompts.
//
// The arithmetic is attn.cu's: codes enter both products as exact FP16 integers,
// the key scale multiplies the finished score, the value scale joins the
// exponent, so that the second product's left operand is 2^(w - m) and
// the denominator takes each 16-key block's sum times 1 / vs.
//
// A CTA takes one or two tiles of 128 query rows (consecutive (token, head of the
// group) pairs of one kv head) and walks the keys they see in tiles of 128:
//  * warps 8..11 unpack: codes from memory into registers one tile ahead, as
//    FP16 integers into shared memory (128-byte swizzle), keys and values in
//    two stages each, and the tile's scales into a small ring.  Values stay [key][d]:
//    the second product reads its right operand with d contiguous (MN-major).
//  * warp 12 issues O_0 += P_0 V, the next S_0 = Q_0 K^T, then the same for row tile 1
//    (O_1 before S_0 where P_1 is there by then): a row tile's softmax runs under the other
//    one's products.
//  * warps 0..3 and 4..7 own a row tile each, a thread a row: scores from tensor
//    memory into registers (which the other warps give up), maximum, 2^x, and the
//    probabilities back over the scores (two FP16 values a column) as the second
//    product's left operand.  The reference m of a row is its maximum as of the last time
//    that mattered: FP16 holds probabilities up to 2^15 as exactly as up to 1, and the
//    denominator is binary32.  So a tile's probabilities are first made about the old
//    reference, without a maximum; only where a row's sum passes 2^15 is the maximum
//    taken, the accumulator rescaled and the tile's probabilities made again.
// Both row tiles share the unpacked keys and values.
//
// Bound by the tensor core, 4 d operations a query row and key: 1.09 PFLOP/s at a prompt of 4,096
// tokens behind 4,096 and one of 395 behind 182, 32 query heads on 8 kv heads of 128 (379 us).
// What stands between: a row tile's scores cannot be made before the product that reads the
// probabilities over them has ended (some 300 cycles each time that nothing else is queued),
// the softmax of 128 x 128 scores takes 1,200 cycles where the two row tiles share the
// schedulers, as much as its products, and the tiles of a grid end unevenly (an eighth).
// With the softmax or the unpacking left out the same call takes 305 or 339 us, with neither 272.
//
// Every wait is bounded (common.cuh): a role that gives up records a timeout and the others follow.
#include "attn_common.cuh"

namespace mnb {

namespace {

constexpr int kSoftWarps = 4;    // a row tile
constexpr int kUnpackWarps = 4;
constexpr int kTileKeys = 128;
constexpr int kTileBlocks = kTileKeys / kKvBlock;
constexpr int kSlab = kTileKeys * 128;  // 128 rows of 64 FP16 values
constexpr int kScaleRing = 4;
constexpr float kMoveBy = 8.f;       // a maximum that grew by no more (log2) stays the reference
constexpr float kMostSum = 32768.f;  // of a row's 128 probabilities: each fits FP16

struct PromptArgs {
    AttnArgs a;
    int64_t units;
    unsigned int* status;
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand in 128-byte swizzled atoms of 8 rows x 128 bytes (1024 bytes apart).
// K-major: the rows are M or N, K runs along the 128 bytes.  MN-major: the rows are K, N
// runs along the 128 bytes and on to the next slab of 64 values, `lead` bytes away.  The low
// word of its descriptor; the high one is the same for all: stride 1024 bytes, version 1,
// 128-byte swizzle.
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand_low(uint32_t saddr, uint32_t lead) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lead ? lead >> 4 : 1u) & 0x3FFFu) << 16;
}

// kind::f16 instruction descriptor: FP32 accumulate, FP16 operands, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool n_major) {
    return (1u << 4) | (n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// The warp that issues stays together and one lane is elected for each product: the operands'
// addresses then stay in uniform registers.  With one lane on a path of its own they are
// moved there for every product, and beside busy warps on the same scheduler a round
// of 32 products took 3,300 cycles instead of 2,200 (2,050 are the tensor core's).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    if (!elected()) return;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kOperandHigh)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    if (!elected()) return;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kOperandHigh)
        : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
    if (!elected()) return;
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 32 columns of this thread's row; the values are there only after landed().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}

// Waits for every tcgen05.ld of the thread; naming the registers keeps their uses behind it.
__device__ __forceinline__ void landed(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])
                 :
                 : "memory");
    asm volatile(""
                 : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// Whether the phase of `parity` is complete.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(bar), "r"(parity)
        : "memory");
    return r != 0;
}

// Bounded wait for it (as mbar_wait), with the plain test first: the wait with a suspend time
// takes 95 cycles even where the phase is complete, the test 15.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned int* status) {
    return bar_test(bar, parity) || mbar_wait(bar, parity, status);
}

// Registers a thread of the calling warpgroup holds from here on.
template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
    return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint4 ldg128(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Pairs of binary32 values in one 64-bit register.
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

template <int D, int NQ>
struct Layout {
    static constexpr int kOperand = D / 64 * kSlab;      // 128 rows of D FP16 values
    static constexpr int kQ = 0;                          // NQ tiles
    static constexpr int kK = kQ + NQ * kOperand;         // two stages
    static constexpr int kV = kK + 2 * kOperand;          // two stages
    static constexpr int kScales = kV + 2 * kOperand;
    static constexpr int kBars = kScales + kScaleRing * kTileBlocks * 16;
    static constexpr int kBytes = kBars + 256 + 1024;     // and the alignment of the swizzle atoms
    // tensor memory: NQ score tiles of 128 columns, then NQ accumulators of D
    static constexpr int kCols = NQ * (128 + D) <= 256 ? 256 : 512;
    // whole warpgroups (the last one issues the products); 128 or 168 registers a thread at
    // launch, dealt out again to softmax, unpacking and the rest
    static constexpr int kThreads = 128 * (NQ + 2);
    static constexpr int kLaunchRegs = NQ == 2 ? 128 : 168;
    static constexpr int kSoftRegs = NQ == 2 ? 176 : 232, kUnpackRegs = NQ == 2 ? 112 : 152, kOtherRegs = NQ == 2 ? 48 : 80;
    static_assert(NQ * kSoftRegs + kUnpackRegs + kOtherRegs <= (NQ + 2) * kLaunchRegs, "within the launch's registers");
};

template <int D, int NQ>
__global__ void __launch_bounds__(Layout<D, NQ>::kThreads, 1) attn_prompt_kernel(const PromptArgs P) {
    using L = Layout<D, NQ>;
    constexpr int kRows = NQ * kPromptTile;
    const AttnArgs& a = P.a;
    unsigned int* status = P.status;
    extern __shared__ unsigned char smem_raw[];
    pdl_wait();

    // later tiles of a sequence see more keys: the long ones of every head start first
    const int head = blockIdx.x % a.b.kv_heads, split = blockIdx.y;
    Tile tl;
    if (!find_tile(a, P.units - 1 - blockIdx.x / a.b.kv_heads, NQ == 1 ? 7 : 8, tl)) return;
    if ((int64_t)tl.n * a.group <= a.skip_rows) return;  // the split kernel's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = (int)min((int64_t)tl.n * a.group - tl.r0, (int64_t)kRows);
    const int first = tl.len - tl.n;
    const int tok_a = tl.r0 / a.group, tok_b = (tl.r0 + rows - 1) / a.group;
    const int hi_t = min(max(first + tok_b + 1, 0), a.b.max_tokens);  // past the table are no keys
    const int lo_t = window_start(a, first + tok_a);
    const int64_t begin64 = (int64_t)(lo_t & ~(kKvBlock - 1)) + (int64_t)split * a.chunk;
    const int begin = (int)min(begin64, (int64_t)hi_t);
    const int end = split == a.splits - 1 ? hi_t : (int)min(begin64 + a.chunk, (int64_t)hi_t);
    const int nj = (int)(((int64_t)end - begin + kTileKeys - 1) / kTileKeys);
    const int all_hi = min(max(first + tok_a + 1, 0), end);
    const int all_lo = window_start(a, first + tok_b);

    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sptr = smem_raw + (base - raw);
    // of a tile's blocks: w = s * .x + .y, denominator += sum * .z
    float4* scales = reinterpret_cast<float4*>(sptr + L::kScales);
    const uint32_t bars = base + L::kBars;
    auto k_full = [&](int s) { return bars + 8u * s; };
    auto k_empty = [&](int s) { return bars + 16u + 8u * s; };
    auto v_full = [&](int s) { return bars + 32u + 8u * s; };
    auto v_empty = [&](int s) { return bars + 48u + 8u * s; };
    auto s_full = [&](int q) { return bars + 64u + 8u * q; };
    auto p_full = [&](int q) { return bars + 80u + 8u * q; };
    auto o_done = [&](int q) { return bars + 96u + 8u * q; };
    const uint32_t q_full = bars + 112u, drain = bars + 120u, tmem_slot = bars + 128u;
    constexpr int kUnpack0 = NQ * kSoftWarps, kMmaWarp = kUnpack0 + kUnpackWarps;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(k_full(s), kUnpackWarps);
            mbar_init(k_empty(s), 1);
            mbar_init(v_full(s), kUnpackWarps);
            mbar_init(v_empty(s), 1);
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), kSoftWarps);
            mbar_init(o_done(s), 1);
        }
        mbar_init(q_full, NQ * kSoftWarps);
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "r"(L::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    // Only now may the next kernel start: the prefill matmul takes its tensor memory before it waits for
    // this one, and must not take it from a CTA that has none yet.  (The registers of these CTAs leave
    // no room for another beside them; this does not rest on that.)
    pdl_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sptr + (tmem_slot - base));

    if (warp >= kMmaWarp) {
        // ---------------------------------------------------------------- products
        give_registers<L::kOtherRegs>();
        if (warp == kMmaWarp) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t q0 = operand_low(base + L::kQ, 0), k0 = operand_low(base + L::kK, 0);
            const uint32_t v0 = operand_low(base + L::kV, kSlab);
            constexpr uint32_t kStep = L::kOperand >> 4;  // descriptors count in 16 bytes
            auto phase = [](int j) { return (uint32_t)(j >> 1) & 1u; };
            // every branch goes by a vote: then the compiler knows that the warp stays together
            auto vote = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };
            auto scores = [&](auto qc, int j) {  // S_q = Q_q K^T of tile j
                constexpr int q = decltype(qc)::value;
                const uint32_t ks = k0 + (uint32_t)(j & 1) * kStep;
                fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (uint32_t)((k / 4 * kSlab + k % 4 * 32) >> 4);
                    mma_ss(tm + q * 128, q0 + q * kStep + off, ks + off, idesc(kTileKeys, false), k > 0);
                }
                commit(s_full(q));
                if (q == NQ - 1) commit(k_empty(j & 1));
            };
            auto add_up = [&](auto qc, int j) {  // O_q += P_q V
                constexpr int q = decltype(qc)::value;
                const uint32_t vs = v0 + (uint32_t)(j & 1) * kStep;
                fence_after();
#pragma unroll
                for (int k = 0; k < kTileKeys / 16; ++k)
                    mma_ts(tm + NQ * 128 + q * D, tm + q * 128 + 8 * k, vs + (uint32_t)(k * 2048 >> 4), idesc(D, true),
                           (j | k) != 0);
                commit(o_done(q));
                if (q == NQ - 1) commit(v_empty(j & 1));
            };
            using First = std::integral_constant<int, 0>;
            using Last = std::integral_constant<int, NQ - 1>;
            bool ok = vote(nj == 0 || bar_wait(q_full, 0, status));
            if (vote(ok && nj > 0)) {
                ok = vote(bar_wait(k_full(0), 0, status));
                if (ok) {
                    scores(First{}, 0);
                    if (NQ == 2) scores(Last{}, 0);
                }
            }
            for (int j = 0; vote(ok && j < nj); ++j) {
                const uint32_t odd = (uint32_t)j & 1u;
                ok = vote(bar_wait(v_full(j & 1), phase(j), status)) && vote(bar_wait(p_full(0), odd, status));
                if (!ok) break;
                add_up(First{}, j);
                const bool more = !vote(j + 1 == nj);
                // The other row tile's probabilities may be there already: then its product runs
                // while this one's end is waited for.
                const bool early = NQ == 2 && vote(bar_test(p_full(NQ - 1), odd));
                if (early) add_up(Last{}, j);
                if (more) {
                    // the probabilities lie over the scores: the product that reads them has to be done
                    ok = vote(bar_wait(k_full((j + 1) & 1), phase(j + 1), status)) && vote(bar_wait(o_done(0), odd, status));
                    if (!ok) break;
                    scores(First{}, j + 1);
                }
                if (NQ == 2) {
                    if (!early) {
                        ok = vote(bar_wait(p_full(NQ - 1), odd, status));
                        if (!ok) break;
                        add_up(Last{}, j);
                    }
                    if (more) {
                        ok = vote(bar_wait(o_done(NQ - 1), odd, status));
                        if (!ok) break;
                        scores(Last{}, j + 1);
                    }
                }
            }
            commit(drain);  // tensor memory is freed only after every issued product has finished
            mbar_wait(drain, 0, status, false);
        }
        __syncwarp();
    } else if (warp >= kUnpack0) {
        // ---------------------------------------------------------------- unpacking
        // A load instruction of the four warps covers 16 rows (D = 128) or 32 (D = 64); the
        // eight lanes of a store phase hold four chunks of two rows, whose swizzled places
        // are eight different 16-byte columns.
        give_registers<L::kUnpackRegs>();
        constexpr int kLoads = D / 16;  // 16-byte pieces a thread and tile
        const int uw = warp - kUnpack0;
        const int chunk = D == 128 ? (lane & 3) + ((lane >> 1) & 4) : lane & 3;
        const int row0 = D == 128 ? uw * 4 + ((lane >> 2) & 1) + ((lane >> 3) & 2) : uw * 8 + (lane >> 2);
        constexpr int kRowsPerLoad = kTileKeys / kLoads;
        const int pmask = (1 << a.b.page_shift) - 1;
        const int lb = lane & (kTileBlocks - 1);  // this lane's block of a tile
        auto block_pos = [&](int j) { return begin + j * kTileKeys + lb * kKvBlock; };
        auto load_page = [&](int j) {
            return j < nj && block_pos(j) < end ? kv_page(a.b, tl.s, block_pos(j)) : -1;
        };
        auto slot_of = [&](int page, int j) {
            return page < 0 ? (int64_t)-1
                            : (((int64_t)page * a.b.kv_heads + head) << a.b.page_shift) + (block_pos(j) & pmask);
        };
        auto load_codes = [&](const uint8_t* codes, int64_t slot, uint4 (&r)[kLoads]) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = i * kRowsPerLoad + row0;
                const int64_t s = __shfl_sync(0xffffffffu, slot, row >> 4);  // the warp's rows lie in one block
                r[i] = s < 0 ? make_uint4(0, 0, 0, 0) : ldg128(codes + (s + (row & 15)) * D + chunk * 16);
            }
        };
        auto store = [&](uint32_t to, const uint4 (&r)[kLoads]) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = i * kRowsPerLoad + row0, c = 2 * chunk;
                const uint32_t at = to + (uint32_t)((c >> 3) * kSlab);
                const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sts128(at + swizzled(row, (c & 7) + h), codes_half2<0x4140u>(w[2 * h]), codes_half2<0x4342u>(w[2 * h]),
                           codes_half2<0x4140u>(w[2 * h + 1]), codes_half2<0x4342u>(w[2 * h + 1]));
            }
        };
        auto wait_empty = [&](uint32_t bar, int j) {  // the warp decides together
            return __all_sync(0xffffffffu, mbar_wait_sleep(bar, ((uint32_t)(j >> 1) & 1u) ^ 1u, status, 32));
        };
        int64_t slot = slot_of(load_page(0), 0);
        int page_next = load_page(1);
        uint4 kc[kLoads], vc[kLoads];
        float ks = 0.f, vs = 1.f;
        if (nj > 0) {
            load_codes(a.K, slot, kc);
            if (slot >= 0) {
                ks = a.Ks[slot >> 4];
                vs = a.Vs[slot >> 4];
            }
        }
        for (int j = 0; j < nj; ++j) {
            const int st = j & 1;
            load_codes(a.V, slot, vc);
            if (!wait_empty(k_empty(st), j)) break;
            store(base + L::kK + st * L::kOperand, kc);
            if (uw == 0 && lane < kTileBlocks) {
                // no such page, or past the end: exponent -infinity, whatever the stage holds
                const float v = vs == 0.f ? 8.67361738e-19f : vs;  // 2^-60: see attn_split_kernel
                scales[(j & (kScaleRing - 1)) * kTileBlocks + lb] =
                    slot < 0 ? make_float4(0.f, -INFINITY, 1.f, 0.f)
                             : make_float4(ks * fabsf(a.scale_log2), __log2f(v), __frcp_rn(v), 0.f);
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_full(st));
            slot = slot_of(page_next, j + 1);
            page_next = load_page(j + 2);
            if (j + 1 < nj) {
                load_codes(a.K, slot, kc);
                ks = slot < 0 ? 0.f : a.Ks[slot >> 4];
                vs = slot < 0 ? 1.f : a.Vs[slot >> 4];
            }
            if (!wait_empty(v_empty(st), j)) break;
            store(base + L::kV + st * L::kOperand, vc);
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full(st));
        }
    } else {
        // ---------------------------------------------------------------- softmax
        take_registers<L::kSoftRegs>();
        const int q = warp / kSoftWarps, sub = warp & 3;  // row tile, quarter of its tensor-memory lanes
        const int r = q * kPromptTile + sub * 32 + lane;  // row of the CTA
        const int tok = (tl.r0 + r) / a.group, qh = head * a.group + (tl.r0 + r - tok * a.group);
        const int64_t trow = tl.row0 + tok;
        const bool ok_row = r < rows && trow >= 0 && trow < a.b.tokens;
        const int pos = first + tok;
        const int hi = ok_row ? min(max(pos + 1, 0), end) : 0;
        const int lo = window_start(a, pos);
        {  // the warp's 32 rows into the operand, 16 bytes a lane, whole rows side by side
            // A negative scale turns the queries' signs instead: a block's largest score then has its
            // largest exponent, whatever the sign.
            const uint32_t turn = a.scale_log2 < 0.f ? 0x80008000u : 0u;
            constexpr int kLanes = D / 8;
            const uint32_t to = base + L::kQ + q * L::kOperand;
            const int c = lane % kLanes;
#pragma unroll 8
            for (int i = 0; i < kLanes; ++i) {
                const int from = i * (32 / kLanes) + lane / kLanes;
                const int64_t at = __shfl_sync(0xffffffffu, ok_row ? trow * a.q_stride + (int64_t)qh * D : -1, from);
                const uint4 v = at >= 0 && nj > 0 ? *reinterpret_cast<const uint4*>(a.Q + at + c * 8) : make_uint4(0, 0, 0, 0);
                sts128(to + (uint32_t)((c >> 3) * kSlab) + swizzled(sub * 32 + from, c & 7), v.x ^ turn, v.y ^ turn, v.z ^ turn,
                       v.w ^ turn);
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const uint32_t lanes = tmem + ((uint32_t)(sub * 32) << 16);
        const uint32_t s_at = lanes + q * 128, o_at = lanes + NQ * 128 + q * D;
        float m = -INFINITY, l = 0.f;  // the reference and the denominator about it
        bool ok = true;

        // One tile of keys; MASK: some row does not see all of it.
        auto tile = [&](int j, auto masked) {
            constexpr bool MASK = decltype(masked)::value;
            const float4* t = scales + (j & (kScaleRing - 1)) * kTileBlocks;
            float x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, x[c]);
            const int p0 = begin + j * kTileKeys;
            auto sees = [&](int i) { return p0 + i < hi && p0 + i >= lo; };
#pragma unroll
            for (int c = 0; c < 4; ++c) landed(x[c]);
            if (MASK) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[c][i] = sees(32 * c + i) ? x[c][i] : -INFINITY;
            }
            float add;  // to the denominator
            // The probabilities about a reference, over the scores (which are in registers); their sum.
            // About a new reference the exponents are rounded as its maximum was, so that none
            // is above it; about the old one in a single step, whose difference from that (half
            // a unit in the last place of the score) only matters where it is so large that the sum tells.
            auto probabilities = [&](float mu, auto fresh) {
                constexpr bool FRESH = decltype(fresh)::value;
                float all = 0.f;
                add = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float4 k = t[2 * c + b];
                        const float lv = FRESH ? k.y : k.y - mu;
                        const uint64_t ks2 = pair(k.x, k.x), lv2 = pair(lv, lv), mu2 = pair(-mu, -mu);
                        uint64_t sum2[2] = {0, 0};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float* y = &x[c][16 * b + 2 * i];
                            uint64_t w2 = fma2(pair(y[0], y[1]), ks2, lv2);
                            if (FRESH) w2 = add2(w2, mu2);
                            float2 w = unpair(w2);
                            w.x = ex2(w.x);
                            w.y = ex2(w.y);
                            if (MASK) {  // a hidden block may have any scale
                                w.x = y[0] == -INFINITY ? 0.f : w.x;
                                w.y = y[1] == -INFINITY ? 0.f : w.y;
                            }
                            sum2[i & 1] = add2(sum2[i & 1], pair(w.x, w.y));
                            p[8 * b + i] = pack_half2(w.x, w.y);
                        }
                        const float2 s = unpair(add2(sum2[0], sum2[1]));
                        const float sum = s.x + s.y;
                        all += sum;
                        if (!MASK || sum != 0.f) add = fmaf(sum, k.z, add);
                    }
                    tmem_st16(s_at + 16 * c, p);
                }
                return all;
            };
            // The reference holds for most tiles: their sum says so.  A row that has none yet, or
            // one that passes it too far (or is NaN), takes the warp through the maximum.
            if (__all_sync(0xffffffffu, m != -INFINITY) && __all_sync(0xffffffffu, probabilities(m, std::false_type{}) <= kMostSum)) {
                l += add;
                return;
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float w = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16; ++i) w = fmaxf(w, x[c][16 * b + i]);
                    top = fmaxf(top, fmaf(w, t[2 * c + b].x, t[2 * c + b].y));
                }
            const bool grown = top > m + kMoveBy || m == -INFINITY;
            const float to = grown ? top : m;
            const float f = grown && m != -INFINITY ? ex2(m - to) : 1.f;
            if (__any_sync(0xffffffffu, f != 1.f)) {  // then j > 0: a tile has been added up
                ok = __all_sync(0xffffffffu, mbar_wait(o_done(q), (uint32_t)(j - 1) & 1u, status));
                if (!ok) return;
                fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(o_at + c, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tmem_st16(o_at + c, o);
                }
                l *= f;
            }
            m = to;
            tmem_wait_st();  // the first try's probabilities go to the same columns
            probabilities(to == -INFINITY ? 0.f : to, std::true_type{});
            l += add;
        };
        for (int j = 0; j < nj; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait(s_full(q), (uint32_t)j & 1u, status));
            if (!ok) break;
            fence_after();
            const int p0 = begin + j * kTileKeys;
            if (p0 >= all_lo && p0 + kTileKeys <= all_hi)
                tile(j, std::false_type{});
            else
                tile(j, std::true_type{});
            if (!ok) break;
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(q));
        }
        if (ok && nj > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(o_done(q), (uint32_t)(nj - 1) & 1u, status));
            fence_after();
        }
        if (ok) {
            const int64_t orow = trow * a.q_heads + qh;
            const float inv = a.splits > 1 ? 1.f : (l == 0.f ? 0.f : __fdiv_rn(1.f, l));
            const bool nothing = nj == 0 || l == 0.f;  // the accumulator holds zeros, or was never written
            // The warp's 32 rows pass through its rows of the query tile (every product that read
            // them is done), kOutBytes of each at a time, so that whole rows are written side by side.
            constexpr int kOutBytes = D == 128 ? 256 : 128;
            constexpr int kOutLanes = kOutBytes / 16;
            const uint32_t mine = base + L::kQ + q * L::kOperand + (uint32_t)(sub * 32 * kOutBytes);
            auto spot = [&](int row, int c) { return mine + (uint32_t)(row * kOutBytes + ((c ^ (row & 7)) << 4)); };
            const bool parts = a.splits > 1;
            const int per = kOutBytes / (parts ? 4 : 2);  // values of a row at a time
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += per) {
#pragma unroll 1
                for (int c = 0; c < per; c += 16) {
                    uint32_t o[16];
                    if (nj > 0) tmem_ld16(o_at + d0 + c, o);
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = nothing ? 0.f : __uint_as_float(o[i]) * inv;
                    if (parts) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sts128(spot(lane, c / 4 + i), __float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                   __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            sts128(spot(lane, c / 8 + i), pack_half2(f[8 * i], f[8 * i + 1]),
                                   pack_half2(f[8 * i + 2], f[8 * i + 3]), pack_half2(f[8 * i + 4], f[8 * i + 5]),
                                   pack_half2(f[8 * i + 6], f[8 * i + 7]));
                    }
                }
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < kOutLanes; ++i) {
                    const int row = i * (32 / kOutLanes) + lane / kOutLanes, c = lane % kOutLanes;
                    char* to = reinterpret_cast<char*>(parts ? reinterpret_cast<uintptr_t>(a.part + (orow * a.splits + split) * D + d0)
                                                             : reinterpret_cast<uintptr_t>(a.out + trow * a.out_stride + (int64_t)qh * D + d0));
                    to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, ok_row ? reinterpret_cast<unsigned long long>(to) : 0ull, row));
                    const uint4 v = lds128(spot(row, c));
                    if (to) *reinterpret_cast<uint4*>(to + c * 16) = v;
                }
                __syncwarp();
            }
            if (ok_row) {
                if (a.splits > 1)
                    *reinterpret_cast<float2*>(a.ml + (orow * a.splits + split) * 2) = make_float2(m, l);
                else if (a.lse)
                    a.lse[orow] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    tmem_wait_st();  // a role that stopped early may have stores in flight
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
}

template <int D, int NQ>
cudaError_t allow() {
    return cudaFuncSetAttribute(attn_prompt_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Layout<D, NQ>::kBytes);
}

template <int D, int NQ>
cudaError_t launch(const PromptArgs& p, cudaStream_t st) {
    return launch_pdl(attn_prompt_kernel<D, NQ>, dim3((unsigned)(p.units * p.a.b.kv_heads), (unsigned)p.a.splits),
                      dim3(Layout<D, NQ>::kThreads), Layout<D, NQ>::kBytes, st, p);
}

}  // namespace

cudaError_t attn_prompt_prepare() {
    cudaError_t e = allow<64, 1>();
    if (e == cudaSuccess) e = allow<64, 2>();
    if (e == cudaSuccess) e = allow<128, 1>();
    if (e == cudaSuccess) e = allow<128, 2>();
    return e;
}

cudaError_t attn_prompt_launch(const AttnArgs& a, int row_tiles, int64_t units, unsigned int* status, cudaStream_t st) {
    const PromptArgs p = {a, units, status};
    if (a.b.head_dim == 64) return row_tiles == 1 ? launch<64, 1>(p, st) : launch<64, 2>(p, st);
    return row_tiles == 1 ? launch<128, 1>(p, st) : launch<128, 2>(p, st);
}

}  // namespace mnb
