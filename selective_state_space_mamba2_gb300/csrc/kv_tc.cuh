// What the tensor-core kernels of attention over pages share: tile sizes, waits, conversions, which keys a row sees, values
// that are not finite.
#pragma once
#include "kv_sched.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace kvtc {

using namespace tc;

constexpr int kRows = 128;    // TMEM lanes: query rows of a tile
constexpr int kKeyShift = 6;
constexpr int kKeys = 1 << kKeyShift;  // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A wait that has to wait, or to look at a limit that may be short.
static __device__ __noinline__ void wait_long(uint64_t *bar, uint32_t parity, volatile int *dead, uint32_t *err, long long limit) {
    const bool spin = limit < 100000;  // a short limit is not slept through
    const long long t0 = clock64();
    while (!(spin ? mbar_test(bar, parity) : mbar_try_wait_sleep(bar, parity, 20000u))) {
        if (*dead) return;
        if (clock64() - t0 > limit) {
            *dead = 1;
            report(err, SSD_DEVERR_TIMEOUT);
            return;
        }
    }
}

struct Waiter {
    volatile int *dead;
    uint32_t *err;
    long long limit;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) const {
        if (!mbar_test(bar, parity)) wait_long(bar, parity, dead, err, limit);
    }
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t f16x2) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four values in two e4m3 parts.
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t &high, uint32_t &low) {
    const uint32_t x = cvt_f16x2(a, b), y = cvt_f16x2(c, d);
    const uint32_t hx = e4m3x2(x), hy = e4m3x2(y);
    high = __byte_perm(hx, hy, 0x5410);
    low = __byte_perm(e4m3x2(sub_f16x2(x, f16x2_of(hx))), e4m3x2(sub_f16x2(y, f16x2_of(hy))), 0x5410);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float log2_of(float v) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// An arrival of this thread on `bar` when the asynchronous copies that it has asked for are done, without being counted up front.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// bits [0, n) set, n clamped to 0 .. 64
__device__ __forceinline__ unsigned long long low_bits(int64_t n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// which keys of tile t the row of new token `tok` sees (tok < 0: no row)
__device__ __forceinline__ unsigned long long seen_bits(const kv_attention_args &a, const kvs::Walk &w, int t, int tok) {
    if (tok < 0) return 0;
    if (t < w.cached_tiles) return low_bits((int64_t)w.q.c - (int64_t)t * kKeys);
    const int base = (t - w.cached_tiles) * kKeys;
    if (!a.tree_mask) return low_bits((int64_t)tok + 1 - base);
    const uint32_t *m = a.tree_mask + (int64_t)(w.q.q0 + tok) * a.mask_words;
    const int word = base / 32;  // base < new tokens <= 32 mask_words
    unsigned long long bits = m[word];
    if (word + 1 < a.mask_words) bits |= (unsigned long long)m[word + 1] << 32;
    return bits & low_bits((int64_t)w.q.n - base);
}

__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t v) {  // mask of the halves whose exponent is all ones
    const uint32_t lo = (v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
    return lo | hi;
}

// The non-finite values that clean_values took out, added to the 32 output columns from `col` of a
// row that sees their keys.
static __device__ __noinline__ void add_nonfinite(const kv_attention_args &a, const kvs::Walk &w, int tok, int col,
                                           uint32_t (&o)[32]) {
    for (int t = max(w.t0, w.cached_tiles); t < w.t1; ++t) {
        const unsigned long long seen = seen_bits(a, w, t, tok);
        const int base = (t - w.cached_tiles) * kKeys;
        for (int j = 0; j < kKeys; ++j) {
            if (!(seen >> j & 1)) continue;
            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_new) +
                                     (int64_t)(w.q.q0 + base + j) * a.v_stride + w.h * a.headdim + col;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float f = to_f32(v[e]);
                if (!isfinite(f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
            }
        }
    }
}

// CTAs that share an item, by a rule on sizes: a pair where the requests have more rows than a tile
// takes on the average, and its two row tiles see the same keys but for one tile of them at most: with a
// mask, or where they are 64 tokens or fewer.  Measured alone / in pairs: 4 prompts of 512 to 4096 tokens
// over up to 8192 cached, 4 query heads to a key head, 771 / 747 to 777 us; 24 trees of 33 to 64 tokens over up
// to 16384, 8 query heads, 209 / 184 to 188 us, of 33 to 48 with 4 heads 297 / 184; 2 times 512 tokens over 65536
// 553 / 444; 64 requests of 1 to 600 over up to 8192 1632 / 1210; but a prompt of 512 tokens beside 64 single
// tokens 187 / 221, since one CTA of the pair then has no rows most of the time.
inline int pair_for(const kv_attention_args &a) {
    const int64_t group = a.nheads / a.kv_heads;
    const bool many = (int64_t)a.total_tokens * group > (int64_t)kRows * a.num_seqs;
    return many && (a.mask_words > 0 || 2 * (kRows / group) <= kKeys) ? 2 : 1;
}

}  // namespace kvtc
}  // namespace ssd
