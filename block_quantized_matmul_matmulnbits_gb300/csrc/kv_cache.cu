// kv_cache.cu -- writing tokens into the 8-bit key/value cache and reading
// them back (mnb_kv_write, mnb_kv_read).
//
// One warp takes one block of 16 positions of one kv head, keys or values: the
// 16 rows that share a scale, 1 or 2 KB of codes that lie together in the
// page.  All of the block's rows are loaded at once (up to eight 16-byte loads
// a lane in flight), the largest magnitude is found with shuffles, and the
// rows go out as 8-byte stores of whole 64- or 128-byte code rows: the tokens
// are read once and nothing waits on another warp.  Both directions are bound
// by memory: 2 bytes in and 1 out a value (written), 1 in and 2 out (read).
// The alternative split, one warp a token, needs the block's scale agreed
// between 16 warps.
//
// Reading 8 kv heads of 128 for 12 sequences of up to 16,384 tokens (356 MB) takes 55.5 us,
// 6.4 TB/s.  Writing and then reading four prompts' 8,146 tokens (100 MB, less than the L2
// cache) takes 19.1 us, 5.2 TB/s: each call loads all there is at once and then
// stores it, and the look for the sequence, its page and its rows comes before.  CTAs of four
// warps: writing and reading a step of 128 sequences took 9.2 us, with eight 10.5, with one
// 10.5; 12.4 instead of 15.6 instructions a value (new_codes below) then made it 8.2, and the
// prompts above 19.1 instead of 20.9.
//
// The magnitude is taken on the FP16 bit patterns without their sign, which
// order as unsigned integers with NaN above infinity above every finite value,
// so a non-finite value reaches the scale without a test of its own.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_batch.cuh"
#include "mnb_internal.h"

namespace mnb {

namespace {

constexpr int kWarps = 4;
constexpr KvSplit kBlocks = {1, 4, 2};  // the blocks of 16 positions that a sequence's tokens touch

struct KvIoArgs {
    KvArgs b;
    int64_t items;
    int64_t row_stride;  // halfs
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    __half *k, *v;
};

// The block of one warp: where its codes and scale lie, and which positions are the call's.
struct KvUnit {
    int which, head;
    int lo, first, end;    // first position of the block; of the call's tokens; the sequence's end in the table
    int64_t row0;          // token row of position `first`
    int64_t slot;          // row of the cache (page, head, row in page) of position lo
};

// False: nothing to do (the whole warp together).
__device__ __forceinline__ bool kv_unit(const KvIoArgs& p, KvUnit& u) {
    const KvArgs& a = p.b;
    const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);  // below 2^32: kv_io
    const unsigned combos = 2u * (unsigned)a.kv_heads;
    const unsigned item = w / combos;
    if (item >= p.items) return false;
    const int c = (int)(w - item * combos);
    u.which = c >= a.kv_heads;
    u.head = u.which ? c - a.kv_heads : c;
    int64_t first_item;
    const KvSeq q = kv_find_seq(a, item, kBlocks, &first_item);
    u.end = min(q.len, a.max_tokens);
    u.first = q.len - q.n;
    u.row0 = q.row0;
    const int64_t lo = ((int64_t)((u.first > 0 ? u.first : 0) >> 4) + ((int64_t)item - first_item)) * kKvBlock;
    if (q.n == 0 || lo < 0 || lo >= u.end) return false;
    u.lo = (int)lo;
    const int page = kv_page(a, q.s, u.lo);
    if (page < 0) return false;
    const int mask = (1 << a.page_shift) - 1;
    u.slot = (((int64_t)page * a.kv_heads + u.head) << a.page_shift) + (u.lo & mask);
    return true;
}

// Two binary32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint2 halves(uint64_t v) {
    uint2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Codes of four new values.  |x * inv| stays below 127.5 (inv is 1 / s to a rounding, and 127 s
// is no less than any of them to another), so nothing has to be clamped; adding 1.5 * 2^23 + 128
// rounds to the nearest integer, ties to even, and leaves the code in the low byte.  The products
// are scalar ones: a packed product and sum become one operation, rounded once, and ties differ.
__device__ __forceinline__ uint32_t new_codes(uint32_t w0, uint32_t w1, float inv) {
    const uint64_t magic = pair(12583040.f, 12583040.f);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w1));
    const uint2 p = halves(add2(pair(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv)), magic));
    const uint2 q = halves(add2(pair(__fmul_rn(b.x, inv), __fmul_rn(b.y, inv)), magic));
    return prmt(prmt(p.x, p.y, 0x0040u), prmt(q.x, q.y, 0x0040u), 0x5410u);
}

// (q - 128) * s of two codes (bytes `sel` of w) as FP16: the code joins the bits of 2^23, which
// is taken off again with the 128.
template <uint32_t LO, uint32_t HI>
__device__ __forceinline__ uint32_t values_half2(uint32_t w, uint64_t s2) {
    const uint64_t t = pair(__uint_as_float(prmt(w, 0x4B000000u, LO)), __uint_as_float(prmt(w, 0x4B000000u, HI)));
    const uint2 v = halves(mul2(add2(t, pair(-8388736.f, -8388736.f)), s2));
    const __half2 h = __floats2half2_rn(__uint_as_float(v.x), __uint_as_float(v.y));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A code of an older token under a scale that grew by 1 / ratio.
__device__ __forceinline__ int quantize_code(float x, float inv) {
    const int c = __float2int_rn(__fmul_rn(x, inv));
    return 128 + (c > 127 ? 127 : (c < -127 ? -127 : c));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const KvIoArgs p) {
    constexpr int LPR = D / 8;          // lanes of a row (8 values each)
    constexpr int RPI = 32 / LPR;       // rows of an iteration
    constexpr int NI = kKvBlock / RPI;  // iterations
    pdl_wait();
    pdl_launch_dependents();
    KvUnit u;
    if (!kv_unit(p, u)) return;
    const int lane = threadIdx.x & 31;
    const int r0 = lane / LPR, c8 = (lane % LPR) * 8;

    const __half* x = (u.which ? p.v : p.k) + (int64_t)u.head * D + c8;
    uint8_t* codes = (u.which ? p.v_codes : p.k_codes) + u.slot * D + c8;
    float* scale = (u.which ? p.v_scales : p.k_scales) + (u.slot >> 4);
    uint4 v[NI];
    unsigned fresh = 0, kept = 0;  // bit i: this lane's row of iteration i is the call's, or older
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int pos = u.lo + i * RPI + r0;
        const int64_t row = u.row0 + (pos - u.first);
        const bool f = pos >= u.first && pos < u.end && row >= 0 && row < p.b.tokens;
        v[i] = f ? *reinterpret_cast<const uint4*>(x + row * p.row_stride) : make_uint4(0, 0, 0, 0);
        fresh |= f ? 1u << i : 0u;
        kept |= pos < u.first ? 1u << i : 0u;
    }
    const bool has_old = u.first > u.lo;
    const float s_old = has_old ? *scale : 0.f;
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        m = __vmaxu2(m, v[i].x & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[i].y & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[i].z & 0x7FFF7FFFu);
        m = __vmaxu2(m, v[i].w & 0x7FFF7FFFu);
    }
    m = max(m & 0xFFFFu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    const float s_new = __fdiv_rn(__half2float(__ushort_as_half((unsigned short)m)), 127.f);
    // fmaxf drops a NaN: the sum keeps it
    const float s = !has_old ? s_new : (s_old != s_old || s_new != s_new) ? s_old + s_new : fmaxf(s_old, s_new);
    const bool good = s > 0.f && s < __int_as_float(0x7f800000);
    const float inv = good ? __fdiv_rn(1.f, s) : 0.f;
    const bool again = has_old && (!good || s != s_old);  // older codes follow the new scale
    const float ratio = again && good ? __fdiv_rn(s_old, s) : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)(i * RPI + r0) * D);
        uint32_t out[2] = {0x80808080u, 0x80808080u};
        if ((fresh >> i) & 1u) {
            if (good) {
                out[0] = new_codes(v[i].x, v[i].y, inv);
                out[1] = new_codes(v[i].z, v[i].w, inv);
            }
            *dst = make_uint2(out[0], out[1]);
        } else if (again && ((kept >> i) & 1u)) {
            if (good) {
                const uint2 q = *dst;
                const uint32_t w[2] = {q.x, q.y};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    out[j] = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float old = (float)((int)((w[j] >> (8 * k)) & 0xFFu) - 128);
                        out[j] |= (uint32_t)quantize_code(old, ratio) << (8 * k);
                    }
                }
            }
            *dst = make_uint2(out[0], out[1]);
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = s;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const KvIoArgs p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, NI = kKvBlock / RPI;
    pdl_wait();
    pdl_launch_dependents();
    KvUnit u;
    if (!kv_unit(p, u)) return;
    const int lane = threadIdx.x & 31;
    const int r0 = lane / LPR, c8 = (lane % LPR) * 8;
    const uint8_t* codes = (u.which ? p.v_codes : p.k_codes) + u.slot * D + c8;
    __half* x = (u.which ? p.v : p.k) + (int64_t)u.head * D + c8;
    uint2 q[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)  // the block's 16 rows are always inside its page
        q[i] = *reinterpret_cast<const uint2*>(codes + (int64_t)(i * RPI + r0) * D);
    const float s = (u.which ? p.v_scales : p.k_scales)[u.slot >> 4];
    const uint64_t s2 = pair(s, s);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int pos = u.lo + i * RPI + r0;
        const int64_t row = u.row0 + (pos - u.first);
        if (pos < u.first || pos >= u.end || row < 0 || row >= p.b.tokens) continue;
        *reinterpret_cast<uint4*>(x + row * p.row_stride) =
            make_uint4(values_half2<0x7440u, 0x7441u>(q[i].x, s2), values_half2<0x7442u, 0x7443u>(q[i].x, s2),
                       values_half2<0x7440u, 0x7441u>(q[i].y, s2), values_half2<0x7442u, 0x7443u>(q[i].y, s2));
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int kv_io(const mnb_kv_cache* c, const mnb_kv_batch* b, void* K, void* V, int64_t row_stride, bool write,
          void* stream) {
    bool empty;
    int rc = kv_check(c, b, &empty);
    if (rc != MNB_OK) return rc;
    if (row_stride < (int64_t)c->kv_heads * c->head_dim) return MNB_ERR_ARG;
    if (row_stride % 8 != 0) return MNB_ERR_ALIGN;
    if (empty || b->max_pages == 0 || c->num_pages == 0) return MNB_OK;
    if (!K || !V) return MNB_ERR_ARG;
    if (!aligned(K, 16) || !aligned(V, 16)) return MNB_ERR_ALIGN;
    KvIoArgs p;
    p.b = kv_args(c, b);
    p.items = kv_items(b->tokens, b->seqs, kBlocks);
    p.row_stride = row_stride;
    p.k_codes = static_cast<uint8_t*>(c->K);
    p.v_codes = static_cast<uint8_t*>(c->V);
    p.k_scales = static_cast<float*>(c->K_scales);
    p.v_scales = static_cast<float*>(c->V_scales);
    p.k = static_cast<__half*>(K);
    p.v = static_cast<__half*>(V);
    const int64_t blocks = (p.items * 2 * c->kv_heads + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX / kWarps) return MNB_ERR_UNSUPPORTED;  // 4 TB of values
    int sms;
    unsigned int* status;
    rc = device_ready(&sms, &status);
    if (rc != MNB_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    const auto kernel = write ? (c->head_dim == 64 ? kv_write_kernel<64> : kv_write_kernel<128>)
                              : (c->head_dim == 64 ? kv_read_kernel<64> : kv_read_kernel<128>);
    return launch_pdl(kernel, grid, block, 0, st, p) == cudaSuccess ? MNB_OK : MNB_ERR_CUDA;
}

}  // namespace

int kv_check(const mnb_kv_cache* c, const mnb_kv_batch* b, bool* empty) {
    if (!c || !b || c->num_pages < 0 || c->kv_heads <= 0 || c->reserved != 0 || b->seqs < 0 || b->max_pages < 0 ||
        b->tokens < 0 || b->max_new < 0 || b->max_len < 0)
        return MNB_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return MNB_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
        return MNB_ERR_UNSUPPORTED;
    if (c->num_pages > INT32_MAX || c->kv_heads > 65535 || b->tokens > INT32_MAX) return MNB_ERR_UNSUPPORTED;
    *empty = b->seqs == 0 || b->tokens == 0;
    if (*empty) return MNB_OK;
    if (!b->kv_len || !b->q_start) return MNB_ERR_ARG;
    // without pages every sequence is empty, and the cache may be NULL
    if (b->max_pages > 0 && c->num_pages > 0 &&
        (!c->K || !c->V || !c->K_scales || !c->V_scales || !b->page_table))
        return MNB_ERR_ARG;
    if (!aligned(c->K, 16) || !aligned(c->V, 16) || !aligned(c->K_scales, 16) || !aligned(c->V_scales, 16) ||
        !aligned(b->page_table, 4) || !aligned(b->kv_len, 4) || !aligned(b->q_start, 4))
        return MNB_ERR_ALIGN;
    return MNB_OK;
}

}  // namespace mnb

extern "C" int mnb_kv_write(const mnb_kv_cache* cache, const mnb_kv_batch* batch, const void* K, const void* V,
                            int64_t row_stride, void* stream) {
    return mnb::kv_io(cache, batch, const_cast<void*>(K), const_cast<void*>(V), row_stride, true, stream);
}

extern "C" int mnb_kv_read(const mnb_kv_cache* cache, const mnb_kv_batch* batch, void* K, void* V,
                           int64_t row_stride, void* stream) {
    return mnb::kv_io(cache, batch, K, V, row_stride, false, stream);
}
