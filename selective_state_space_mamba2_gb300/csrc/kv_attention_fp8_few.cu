// kv_tree_attention_fp8 on the tensor cores for row tiles of at most 32 rows (decode steps, short drafts): a cache in 8
// bits, tokens in bf16, headdim 64 or 128.
//
// With few query rows the keys are the long side, so they are the rows of the products (TMEM lanes), in tiles of 128:
//   S^T = K Q^T        e4m3, 128 x 2R, K = headdim: the codes as they are; queries as two parts, high and low, side by side
//   P   = 2^(t - m)    t = s (c / u) ks + log2 vs; one key per thread, its R weights as four e5m2 parts to shared memory
//   O^T += V^T P       e4m3 times e5m2, headdim x 4R, K = 128: all parts at once, each to its own columns
// R is 16 or 32.  A key's scales ks, vs are constants of its thread; u is the row's unit, the power of two that puts its
// largest query entry in [128, 256).  A tile's codes are read once for each product, 16 KB and 16 KB, whatever the rows
// (with the queries as rows, padded to 128 of them, a product read them, too: 642 cycles of an SM for 64 keys, here 352 for
// 128), and a thread has R weights to make for 128 keys, not 64 for 64.
//
// m belongs to a row.  It is 2^12 below the row's largest weight when it is set, and a tile is taken by it as long as no
// weight passes 2^15 (fp16 ends at 2^16), which the threads find out by one barrier that votes; only where one does (an
// item's first tile, seldom later) the maxima are reduced, and O^T and the sums rescaled.  A value's scale is part of its
// weight; the sum of the weights takes them without, divided by it.  A weight below 2^-126 is lost to both: with scales of a request
// at most 2^96 apart, it is 2^-42 of the largest or less.  Sums stay with the threads, a row's 128 of them are added up at the end.
//
// Rounding.  Queries in two parts lose at most 2^-17 of the row's largest entry (kv_attention_fp8_tc.cu).  Weights are
// rounded to fp16: off by 2^-11 of themselves, or 2^-37 of the largest that m was set by.  e5m2 is fp16 without its last 8
// bits, so a part takes a weight's first three significant bits as they stand, and the next one what is left times 8: the four,
// in units of 1, 1/8, 1/64 and 1/512, hold an fp16 number exactly, down to its smallest step.  (Two e4m3 parts reach
// only 2^-17 below the largest weight: beside one key with 0.9 of it 8192 others lost 5 % of theirs, with 0.97 40 %.)
//
// New tokens' tiles are bf16 with the queries as they were given: 64-column halves of 128 keys, and 64 keys' values, in a
// ring stage each; weights as two bf16 parts.
//
// What bounds it: HBM for large batches (256 requests of 4 tokens over up to 8192 in blocks of 64, 2.27 GB, 385 to 398 us, 0.84
// to 0.87 of the copy rate; a 16-bit cache 664 us), the softmax warps' instructions with tiles of 32 rows (64 requests of 8 tokens, 4
// query heads to a key head, over up to 8192: 182 us; 164 with two e4m3 parts, 7 instructions for two weights instead of
// 12), latency for one token over 777 (14.5 us with the join).  With weights in two e4m3 parts, on the first of these:
// queries as rows, padded to 128 of them, 603 us; three CTAs to an SM 416; every CTA with heads of its own choice 535; now 391.
//
// Masked places: a weight that must not count is set to 0, whatever its score is.  Values' rows that are not there
// are zeroed in shared memory; new tokens' values that are not finite are taken out and added at the end.  Waits are bounded as in
// kv_attention_tc.cu.
#include "kv_fp8.cuh"
#include "kv_tc.cuh"
#include "tmap.h"

namespace ssd {
namespace {

using namespace tc;
using fp8::max_u16x2;
using kvtc::copies_arrive;
using kvtc::copy4;
using kvtc::cvt_f16x2;
using kvtc::ex2;
using kvtc::kLn2;
using kvtc::kLog2e;
using kvtc::log2_of;
using kvtc::max3;
using kvtc::nonfinite_bf16x2;
using kvtc::reciprocal;
using kvtc::split4;
using kvtc::sub_f16x2;
using kvtc::Waiter;

constexpr int kThreads = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kKeyShift = 7, kKeys = 1 << kKeyShift;
constexpr int kOverhead = 2;          // of an item, in key tiles
constexpr int kScaleRing = 4;         // tiles whose scales are kept: the ring lets keys come three tiles ahead
constexpr int kStage = kKeys * 128;   // bytes of a ring stage
constexpr int kBoxes = kKeys / 8;     // most boxes of a tile
constexpr float kBelow = 12.f;        // m is so far (base 2) below the largest weight when it is set
constexpr float kMost = 15.f;         // weights stay at most 2^15
constexpr float kSlack = 2.f;         // of the rows whose m could be set, those are that have grown by so much
constexpr int kPieces = 4;            // e5m2 parts of a weight
constexpr float kUnit = 8.f;          // of a part, against the next one
constexpr uint32_t kSoftmaxBar = 1, kVoteBar = 2;

struct Params {
    kv_attention_args a;
    const float *k_scale, *v_scale;
    kvs::Parts parts;
    kvs::Tiling g;
    uint32_t group_inv;          // ceil(2^16 / query heads per key head): row / group = row * group_inv >> 16
    int32_t box_shift;           // rows of a page that one copy brings: a power of two that divides block_size and kKeys
    int32_t key_shift, val_shift;  // rows of new tokens that one copy of keys, of values brings
    long long wait_limit;
};

template <int R> constexpr int kStages = R == 16 ? 5 : 4;

template <int R> struct Bars {
    enum {
        Q_FULL, Q_EMPTY, QP_READY, S_FULL0, S_FULL1, P_READY0, P_READY1, O_DONE0, O_DONE1, FIN, SCALES0,
        KV_FULL0 = SCALES0 + kScaleRing, KV_EMPTY0 = KV_FULL0 + kStages<R>, NUM = KV_EMPTY0 + kStages<R>
    };
};

template <int D, int R> struct Layout {
    static constexpr int kParts = 0;                              // [2R] rows of D bytes: high parts, low parts
    static constexpr int kQ = kParts + 2 * R * D;                 // queries: [D / 64][R] rows of 128 bytes
    static constexpr int kP = kQ + R * D * 2;                     // weights: [128] rows of 4R bytes, a part after the other
                                                                  // (of new tokens: two tiles of 2R bytes, high and low parts)
    static constexpr int kRing = kP + kKeys * kPieces * R;
    static constexpr int kScales = kRing + kStages<R> * kStage;   // [kScaleRing][2][kBoxes]: ks, vs of a tile's boxes
    static constexpr int kFactors = kScales + kScaleRing * 2 * kBoxes * 4;  // [2][R]: c / u of an item's rows
    static constexpr int kTops = kFactors + 2 * R * 4;            // [R]: m
    static constexpr int kShrink = kTops + R * 4;                 // [R]: what O^T and the sums are multiplied by
    static constexpr int kRed = kShrink + R * 4;                  // [4 warps][R]
    static constexpr int kBars = kRed + 4 * R * 4;
    static constexpr int kMisc = kBars + Bars<R>::NUM * 8;        // TMEM base, dead mark, items with non-finite values
    static constexpr int kBytes = kMisc + 16;
    static constexpr int kFind = kRing;                           // before the ring is used
    static_assert(kRing % 1024 == 0 && kP % 1024 == 0 && kQ % 1024 == 0, "swizzled tiles");
    static_assert(kBytes <= 113 * 1024, "two CTAs to an SM");
};

// byte offset of 16-byte piece c of row r in a tile of rows of `width` bytes, swizzled over them
template <int width> __device__ __forceinline__ uint32_t row_offset(uint32_t r, uint32_t c) {
    return width == 128 ? sw128_offset(r, c) : width == 64 ? sw64_offset(r, c) : sw32_offset(r, c);
}
template <int width> __device__ __forceinline__ uint64_t row_desc(const void *p, uint32_t lbo) {  // 8 rows and on
    const uint32_t at = smem_u32(p);
    return width == 128 ? sw128_desc(at, lbo, 1024) : width == 64 ? sw64_desc(at, lbo, 512) : sw32_desc(at, lbo, 256);
}

// Four weights, as fp16, in e5m2 parts: an fp16 number's first byte, and the rest times 8 (neither rounds).
__device__ __forceinline__ void pieces4(float2 a, float2 b, uint32_t (&part)[kPieces]) {
    constexpr uint32_t kFirst = 0xFF00FF00u, kEight = 0x48004800u;  // first bytes; 8, twice
    uint32_t x = cvt_f16x2(a.x, a.y), y = cvt_f16x2(b.x, b.y);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        part[i] = __byte_perm(x, y, 0x7531);
        if (i + 1 == kPieces) break;
        x = hmul2_u32(sub_f16x2(x, x & kFirst), kEight);
        y = hmul2_u32(sub_f16x2(y, y & kFirst), kEight);
    }
}

// Whether any of the softmax threads says so; all of them call it.
__device__ __forceinline__ bool vote(bool mine) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(any)
                 : "r"((uint32_t)mine), "n"(kVoteBar)
                 : "memory");
    return any != 0;
}
template <int N> __device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[N]) {
    if constexpr (N == 16)
        tmem_ld16(at, r);
    else if constexpr (N == 32)
        tmem_ld32(at, r);
    else
        tmem_ld64(at, r);
}
// Over the warp, the sum (or the largest, NaN aside) of each of R values a lane; lane i gets that of row i * R / 32.
template <int R, bool kMax> __device__ __forceinline__ float over_warp(float (&v)[R], int lane) {
    int n = R;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                if (i >= n) break;
                const bool up = lane & o;
                const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                const float got = __shfl_xor_sync(~0u, send, o);
                v[i] = kMax ? fmaxf(keep, got) : keep + got;
            }
        } else {
            const float got = __shfl_xor_sync(~0u, v[0], o);
            v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return v[0];
}

// The queries as two e4m3 parts and their rows' c / u, by the four softmax warps: a row by 32 (D = 64: 16) lanes, 4 entries
// each.  Rows that are not there are zeros.
template <int D, int R> __device__ __forceinline__ void split_queries(uint8_t *smem, int rows, float c, float *factors, int warp,
                                                                      int lane) {
    using L = Layout<D, R>;
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;
    const int sub = lane % kLanes, mine = lane / kLanes;
#pragma unroll
    for (int i = 0; i < R / (4 * kAtOnce); ++i) {
        const int row = (i * 4 + warp) * kAtOnce + mine;
        uint2 x = *reinterpret_cast<const uint2 *>(smem + L::kQ + (sub >> 4) * (R * 128) + sw128_offset(row, sub >> 1 & 7) + (sub & 1) * 8);
        if (row >= rows) x = make_uint2(0, 0);
        uint32_t top = max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        // magnitudes of bf16 compare as whole numbers; NaN and infinity are larger than any
        const int e = (int)(top >> 7);  // biased exponent
        float unit = __uint_as_float((uint32_t)min(134 + 127 - e, 254) << 23);
        if (e == 255) unit = __uint_as_float(0x7FC00000u);  // the row's scores are NaN
        if (top == 0) unit = 1.f;
        uint32_t hi, lo;
        split4(__uint_as_float(x.x << 16) * unit, __uint_as_float(x.x & 0xFFFF0000u) * unit, __uint_as_float(x.y << 16) * unit,
               __uint_as_float(x.y & 0xFFFF0000u) * unit, hi, lo);
        uint8_t *to = smem + L::kParts;
        *reinterpret_cast<uint32_t *>(to + row_offset<D>(row, sub >> 2) + (sub & 3) * 4) = hi;
        *reinterpret_cast<uint32_t *>(to + row_offset<D>(R + row, sub >> 2) + (sub & 3) * 4) = lo;
        if (sub == 0) factors[row] = c / unit;
    }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2)
    kv_attention_fp8_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKc,
                                const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmKn,
                                const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Layout<D, R>;
    using B = Bars<R>;
    constexpr int kHalves = D / 64, kRing = kStages<R>;
    constexpr uint32_t kTmemCols = R == 16 ? 128 : 256;
    constexpr uint32_t COL_S = 0, COL_O = 4 * R;  // two score tiles of 2R columns, the output's 4R
    static_assert(kTmemCols == 4 * R + kPieces * R, "columns");
    const kv_attention_args &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int group = a.nheads / a.kv_heads;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *dead = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    volatile int *dirty = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);

    launch_dependents();  // the join kernel may be set up as CTAs of this one end
    if (warp == kMmaWarp) {  // tensor memory first: see kv_attention_tc.cu
        tmem_alloc(sTmem, kTmemCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmKc);
        tma_prefetch_desc(&tmVc);
        tma_prefetch_desc(&tmKn);
        tma_prefetch_desc(&tmVn);
        for (int i = 0; i < B::NUM; ++i)
            mbar_init(&bar[i], i == B::P_READY0 || i == B::P_READY1 || i == B::QP_READY ? 4
                               : i >= B::SCALES0 && i < B::SCALES0 + kScaleRing          ? kBoxes
                                                                                         : 1);
        fence_mbar_init();
        *dead = 0;
        dirty[0] = dirty[1] = 0;
    }
    kvs::Walk w;
    // Workers of all heads side by side: CTAs of different heads walk over the same blocks at about the same time, so that
    // a row of a block, all heads' keys of a token, is read from HBM in one go.
    const int head = blockIdx.x % a.kv_heads, run = blockIdx.x / a.kv_heads, runs = gridDim.x / a.kv_heads, worker = head * runs + run;
    const bool work = kvs::find_run<true>(a, p.g, run, runs, *reinterpret_cast<kvs::FindSmem *>(smem + L::kFind),
                                          p.parts.borders + head * runs, w, head);
    const bool aligned = (smem_u32(smem) & 1023u) == 0;  // the swizzled tiles need a 1024-byte aligned base
    if (!aligned && tid == 0) report(a.err_word, SSD_DEVERR_INTERNAL);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *sTmem;
    const Waiter wait{dead, a.err_word, p.wait_limit};

    if (!work || !aligned) {
        // nothing to do
    } else if (warp == kLoadWarp) {
        // ---- loads -----------------------------------------------------------------
        // A cached tile comes in boxes of rows of one block, 1 to 16 of them: the first 16 lanes ask for keys, a box each,
        // and for the box's scales; the others for values, one tile behind, as the ring's order is.
        uint32_t st = 0, phase = 0;  // ring stage, its phase
        uint32_t items = 0, tile = 0;
        uint32_t asked = 0, asked_q = 0;  // stages and query tiles whose copies were asked for: all up to a wait that gave up
        struct Page {
            int32_t col, off, id;
        };
        const int my_box = lane & 15, role = lane >> 4;  // 0: keys, 1: values
        const int row0 = my_box << p.box_shift;          // of the tile
        const bool mine = row0 < kKeys;
        const int step = kKeys / a.block_size, step_off = kKeys % a.block_size;
        // This lane's page of cached tile t; its block id is read a tile ahead (kv_attention_tc.cu).
        auto page = [&](int32_t col, int32_t off, int t) {
            Page g{col, off, 0};
            if (t < w.cached_tiles && mine && (int64_t)t * kKeys + row0 < w.q.c)
                g.id = a.block_table[(int64_t)w.r * a.table_cols + col];
            return g;
        };
        auto page_of = [&](int t) {
            const int32_t pos = t * kKeys + row0;
            return page(pos / a.block_size, pos % a.block_size, t);
        };
        auto page_after = [&](const Page &g, int t) {
            const int32_t off = g.off + step_off;
            const bool over = off >= a.block_size;
            return page(g.col + step + over, over ? off - a.block_size : off, t);
        };
        auto stage_after = [&](uint32_t s) { return s + 1 == kRing ? 0 : s + 1; };
        bool gave_up = false;
        // Waits until stage `s` is free; false where a wait gave up, anyone's, now or before: nothing is asked for after that.
        // (A stage counts as free, too, where the products did not wait for its copies, which then are still on their way.)
        auto is_free = [&](uint32_t s, uint32_t parity) {
            if (gave_up) return false;
            wait(&bar[B::KV_EMPTY0 + s], parity);
            gave_up = __any_sync(~0u, *dead);
            return !gave_up;
        };
        // This lane's box of cached tile t into stage s.
        auto ask = [&](uint32_t s, int t, const Page &g) {
            const int boxes = (min(kKeys, w.q.c - t * kKeys) + (1 << p.box_shift) - 1) >> p.box_shift;
            uint64_t *full = &bar[B::KV_FULL0 + s];
            if (my_box == 0) mbar_arrive_expect_tx(full, (boxes * D) << p.box_shift);
            if (my_box < boxes) {
                int32_t id = g.id;
                if (id < 0 || id >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    id = a.num_blocks;  // outside the tensor: reads as zeros
                }
                tma_load_4d(smem + L::kRing + s * kStage + row0 * D, role ? &tmVc : &tmKc, 0, g.off, w.h, id, full);
            }
        };
        // The next stage(s) for tile t's keys or values alone.
        auto load = [&](bool value, int t, const Page &g) {
            const bool cached = t < w.cached_tiles;
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
                if (i > 0 && cached) break;
                const uint32_t s = st;
                const bool ok = is_free(s, phase ^ 1);
                if ((st = stage_after(st)) == 0) phase ^= 1;
                if (!ok) return;
                ++asked;
                uint64_t *full = &bar[B::KV_FULL0 + s];
                uint8_t *dst = smem + L::kRing + s * kStage;
                const int base = (t - w.cached_tiles) * kKeys, left = w.new_seen - base;  // of new tokens
                if (cached) {
                    if (role == (int)value) ask(s, t, g);
                } else if (!value || kHalves == 1) {  // columns 64 i on of all keys (values of 64 columns: the same)
                    const int shift = value ? p.val_shift : p.key_shift;
                    const int boxes = (min(kKeys, left) + (1 << shift) - 1) >> shift;
                    if (lane == 0) mbar_arrive_expect_tx(full, (boxes * 128) << shift);
                    if (lane < boxes)
                        tma_load_4d(dst + (lane << shift) * 128, value ? &tmVn : &tmKn, 0, w.q.q0 + base + (lane << shift), i, w.h,
                                    full);
                } else {  // both halves of the columns of keys 64 i on
                    const int shift = p.val_shift, at = lane & 15, half = lane >> 4;
                    const int boxes = (min(64, max(0, left - 64 * i)) + (1 << shift) - 1) >> shift;
                    if (lane == 0) mbar_arrive_expect_tx(full, (boxes * kHalves * 128) << shift);
                    if (at < boxes)
                        tma_load_4d(dst + half * 8192 + (at << shift) * 128, &tmVn, 0, w.q.q0 + base + 64 * i + (at << shift), half,
                                    w.h, full);
                }
                __syncwarp();
            }
        };
        // Keys of cached tile t and values of the one before it, into the next two stages.
        auto load_both = [&](int t, const Page &g) {
            const uint32_t s0 = st, s1 = stage_after(s0), phase1 = s1 == 0 ? phase ^ 1 : phase;
            st = stage_after(s1);
            const bool ok = is_free(role ? s1 : s0, (role ? phase1 : phase) ^ 1);
            phase = st == 0 || s1 == 0 ? phase ^ 1 : phase;
            if (!ok) return;
            asked += 2;
            ask(role ? s1 : s0, t - role, g);
            __syncwarp();
        };
        // Scales of cached tile's blocks to their place in shared memory, a pair for each box; each of 16 lanes arrives on
        // the tile's barrier when its copies are done.  The place is free: a tile's scales are read before its weights
        // are written, and the ring only lets keys come in a few tiles further on.
        auto load_scales = [&](int t, const Page &g) {
            if (gave_up || t >= w.cached_tiles) return;
            if (role == 0) {
                float *to = reinterpret_cast<float *>(smem + L::kScales) + (tile % kScaleRing) * 2 * kBoxes + my_box;
                uint64_t *full = &bar[B::SCALES0 + tile % kScaleRing];
                if (mine && t * kKeys + row0 < w.q.c && g.id >= 0 && g.id < a.num_blocks) {
                    const int64_t at = (int64_t)g.id * a.kv_heads + w.h;
                    copy4(to, p.k_scale + at);
                    copy4(to + kBoxes, p.v_scale + at);
                    copies_arrive(full);
                } else {
                    to[0] = to[kBoxes] = 1.f;
                    mbar_arrive(full);
                }
            }
            ++tile;
            __syncwarp();
        };
        bool more = true;
        while (more) {
            Page now = page_of(w.t0);  // of tile t for keys, of tile t - 1 for values (from the second one on)
            wait(&bar[B::Q_EMPTY], (items & 1) ^ 1);
            ++items;
            if (!__any_sync(~0u, *dead)) {
                asked_q = items;
                if (lane == 0) mbar_arrive_expect_tx(&bar[B::Q_FULL], kHalves * p.g.tokens * group * 128);
                __syncwarp();
                if (lane < kHalves)
                    tma_load_3d(smem + L::kQ + lane * (R * 128), &tmQ, lane * 64, w.h * group, w.q.q0 + w.first_token(p.g),
                                &bar[B::Q_FULL]);
            }
            __syncwarp();
            for (int t = w.t0; t < w.t1; ++t) {
                Page next = now;  // of a tile further on, read ahead; values start a tile later
                if (role == 0 || t > w.t0) next = page_after(now, t + 1 - role);
                if (t == w.t0) {
                    load(false, t, now);
                } else if (t < w.cached_tiles) {
                    load_both(t, now);
                } else {
                    load(false, t, now);
                    load(true, t - 1, now);
                }
                load_scales(t, now);
                now = next;
            }
            load(true, w.t1 - 1, now);
            more = w.next<true>(a, p.g);
        }
        // The copies asked for land before the CTA may go, whether a wait gave up before the last was asked for, gives
        // up after it, or none does (then the products have waited for them).
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (uint32_t k = 0; k < kRing && k < asked; ++k)
            mbar_wait(&bar[B::KV_FULL0 + (asked - 1 - k) % kRing], (asked - 1 - k) / kRing & 1, 20000000ll);
        if (asked_q > 0) mbar_wait(&bar[B::Q_FULL], (asked_q - 1) & 1, 20000000ll);
    } else if (warp == kMmaWarp) {
        // ---- products --------------------------------------------------------------
        // In the order of kv_attention_tc.cu, and as there: the warp walks along, an elected lane issues from uniform
        // values, and a wait that gave up does not stop it.
        const uint32_t tmu = __shfl_sync(~0u, tm, 0);
        constexpr uint32_t kIdS8 = idesc_e4m3(128, 2 * R, 0, 0), kIdO8 = idesc_e4m3_e5m2(128, kPieces * R, 1, 1);
        constexpr uint32_t kIdS = idesc_bf16(128, R, 0, 0), kIdO = idesc_bf16(128, R, 1, 1);
        // values of 64 columns: their columns twice (the second 64 rows of O^T are not used)
        const uint64_t dParts = row_desc<D>(smem + L::kParts, 16), dQ = row_desc<128>(smem + L::kQ, 16);
        const uint64_t dK8 = row_desc<D>(smem + L::kRing, 16), dV8 = row_desc<D>(smem + L::kRing, 0);
        const uint64_t dK = row_desc<128>(smem + L::kRing, 16), dV = row_desc<128>(smem + L::kRing, kHalves == 2 ? 8192 : 0);
        const uint64_t dP8 = row_desc<kPieces * R>(smem + L::kP, 0), dP = row_desc<2 * R>(smem + L::kP, 0);
        uint32_t st = 0, phase = 0;  // ring stage and its phase
        uint32_t tile = 0, items = 0, split = 0;  // split: items whose queries were split
        auto take = [&]() {  // waits for the next stage; its number, uniform
            wait(&bar[B::KV_FULL0 + st], phase);
            const uint32_t s = __shfl_sync(~0u, st, 0);
            if (++st == kRing) st = 0, phase ^= 1;
            return s;
        };
        auto scores = [&](uint32_t g, bool cached, bool last) {  // of tile number g, the item's last or not
            const uint32_t s0 = take(), s1 = !cached && kHalves > 1 ? take() : s0;
            tc_fence_after();
            const uint32_t gg = __shfl_sync(~0u, g, 0);
            const uint32_t d = tmu + COL_S + 2 * R * (gg & 1);
            if (elect_one()) {
                if (cached) {
                    const uint64_t k0 = desc_at(dK8, s0 * kStage);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) mma8_ss(d, desc_at(k0, 32 * k), desc_at(dParts, 32 * k), kIdS8, k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(d, desc_at(dK, (k >> 2 ? s1 : s0) * kStage + (k & 3) * 32),
                               desc_at(dQ, (k >> 2) * (R * 128) + (k & 3) * 32), kIdS, k > 0);
                }
                mma_commit(&bar[B::S_FULL0 + (gg & 1)]);
                mma_commit(&bar[B::KV_EMPTY0 + s0]);
                if (kHalves > 1 && !cached) mma_commit(&bar[B::KV_EMPTY0 + s1]);
                if (last) mma_commit(&bar[B::Q_EMPTY]);
            }
            __syncwarp();
        };
        auto output = [&](uint32_t g, bool cached, uint32_t add) {  // of tile number g
            const uint32_t s0 = take(), s1 = !cached && kHalves > 1 ? take() : s0;
            const uint32_t gg = __shfl_sync(~0u, g, 0);
            wait(&bar[B::P_READY0 + (g & 1)], (g >> 1) & 1);
            tc_fence_after();
            if (elect_one()) {
                if (cached) {
                    const uint64_t v0 = desc_at(dV8, s0 * kStage);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma8_ss(tmu + COL_O, desc_at(v0, 32 * D * k), desc_at(dP8, 32 * kPieces * R * k), kIdO8, k > 0 ? 1u : add);
                } else {
                    // 64 keys in a stage, or all 128 of 64 columns; high parts to the first columns, low ones to the next
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ss(tmu + COL_O + R * part, desc_at(dV, (kHalves > 1 && k > 3 ? s1 * kStage + 2048 * (k - 4) : s0 * kStage + 2048 * k)),
                                   desc_at(dP, part * (kKeys * 2 * R) + 32 * R * k), kIdO, k > 0 ? 1u : add);
                }
                mma_commit(&bar[B::O_DONE0 + (gg & 1)]);
                mma_commit(&bar[B::KV_EMPTY0 + s0]);
                if (kHalves > 1 && !cached) mma_commit(&bar[B::KV_EMPTY0 + s1]);
            }
            __syncwarp();
        };
        bool more = true;
        while (more) {
            const int n = __shfl_sync(~0u, w.t1 - w.t0, 0), cached = __shfl_sync(~0u, w.cached_tiles - w.t0, 0);
            wait(&bar[B::Q_FULL], items & 1);
            ++items;
            if (cached > 0) {
                wait(&bar[B::QP_READY], split & 1);
                ++split;
            }
            scores(tile, cached > 0, n == 1);
            for (int i = 1; i < n; ++i) {
                scores(tile + i, i < cached, i == n - 1);
                output(tile + i - 1, i - 1 < cached, i > 1);
            }
            output(tile + n - 1, n - 1 < cached, n > 1);
            tile += n;
            more = w.next<true>(a, p.g);
        }
        if (elect_one()) mma_commit(&bar[B::FIN]);  // everything issued is done before the CTA goes
        mbar_wait(&bar[B::FIN], 0, 20000000ll);
        __syncwarp();
    } else {
        // ---- softmax and output: a thread has a key of each tile, at the end a column of the output -----
        const float c = a.scale * kLog2e;
        const uint32_t lane_base = tm + ((uint32_t)(warp * 32) << 16);
        const float *scales = reinterpret_cast<const float *>(smem + L::kScales);
        float *tops = reinterpret_cast<float *>(smem + L::kTops), *shrinks = reinterpret_cast<float *>(smem + L::kShrink);
        float *red = reinterpret_cast<float *>(smem + L::kRed);
        uint32_t tile = 0, ring = 0, scaled = 0;  // tile number, ring stages used by earlier items, cached tiles
        int item = 0;
        auto factors_of = [&](int i) { return reinterpret_cast<float *>(smem + L::kFactors) + (i & 1) * R; };
        auto rows_of = [&](const kvs::Walk &v) { return v.tokens(p.g) * group; };
        // The queries of item number i in parts, if it has cached tiles.  The scores of the item before are done.
        auto split = [&](const kvs::Walk &v, int i) {
            if (v.t0 >= v.cached_tiles) return;
            wait(&bar[B::Q_FULL], i & 1);
            __syncwarp();
            split_queries<D, R>(smem, rows_of(v), c, factors_of(i), warp, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B::QP_READY]);
        };
        split(w, 0);
        bool more = true;
        while (more) {
            const float *factors = factors_of(item);
            ++item;
            const int token0 = w.first_token(p.g), rows = rows_of(w), n_tiles = w.t1 - w.t0;
            const uint32_t row_bits = rows >= 32 ? ~0u : (1u << rows) - 1;
            const int pieces = w.t0 < w.cached_tiles ? kPieces : 2;  // columns of O^T that are in use, in parts
            // ring stages of the item's first x tiles
            auto stages = [&](int x) { return x + (kHalves - 1) * max(0, x - max(0, w.cached_tiles - w.t0)); };
            // which rows see new token j
            auto seen_by = [&](int j) -> uint32_t {
                if (j >= w.new_seen) return 0;
                if (!a.tree_mask) {
                    const int first = (j - token0) * group;  // row
                    return first <= 0 ? row_bits : first >= rows ? 0u : row_bits & (~0u << first);
                }
                uint32_t bits = 0;
                const uint32_t one = group >= 32 ? ~0u : (1u << group) - 1;
                for (int i = 0; i * group < rows; ++i) {
                    const uint32_t *m = a.tree_mask + (int64_t)(w.q.q0 + token0 + i) * a.mask_words;
                    if (m[j >> 5] >> (j & 31) & 1) bits |= one << (i * group);
                }
                return bits;
            };
            if (tid < R) tops[tid] = -INFINITY;
            named_bar_sync(kSoftmaxBar, 128);
            float2 sum[R / 2];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) sum[r] = make_float2(0.f, 0.f);
            for (int t = w.t0; t < w.t1; ++t, ++tile) {
                const bool cached = t < w.cached_tiles;
                const uint32_t s_col = lane_base + COL_S + 2 * R * (tile & 1);
                const int base = (cached ? t : t - w.cached_tiles) * kKeys;
                const uint32_t seen = cached ? (base + tid < w.q.c ? ~0u : 0u) : seen_by(base + tid);
                float f = c, shift = 0.f, inv = 1.f;  // scores in base 2 are s f factor + shift; a weight counts inv times
                if (cached) {
                    wait(&bar[B::SCALES0 + scaled % kScaleRing], scaled / kScaleRing & 1);
                    const float *sc = scales + (scaled % kScaleRing) * 2 * kBoxes + (tid >> p.box_shift);
                    const float vs = sc[kBoxes];
                    f = sc[0], shift = log2_of(vs), inv = reciprocal(vs);  // exact for powers of two, else off by 2^-22
                    ++scaled;
                }
                wait(&bar[B::S_FULL0 + (tile & 1)], (tile >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                float2 x[R / 2];
                if (cached) {
                    uint32_t s[2 * R];
                    tmem_ld<2 * R>(s_col, s);
                    tmem_ld_wait();
#pragma unroll
                    for (int r = 0; r < R / 2; ++r)
                        x[r] = add_f2(make_float2(__uint_as_float(s[2 * r]), __uint_as_float(s[2 * r + 1])),
                                      make_float2(__uint_as_float(s[R + 2 * r]), __uint_as_float(s[R + 2 * r + 1])));
                } else {
                    uint32_t s[R];
                    tmem_ld<R>(s_col, s);
                    tmem_ld_wait();
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) x[r] = make_float2(__uint_as_float(s[2 * r]), __uint_as_float(s[2 * r + 1]));
                }
                // scores in base 2, a value's scale with them
#pragma unroll
                for (int r = 0; r < R / 2; ++r) {
                    float2 k = make_float2(f, f);
                    if (cached) k = mul_f2(k, *reinterpret_cast<const float2 *>(factors + 2 * r));
                    x[r] = fma_f2(x[r], k, make_float2(shift, shift));
                }
                float2 v[R / 2];
                float over = -INFINITY;  // by how much the largest is above the row's m
                auto weigh = [&]() {
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) {
                        const float2 m = *reinterpret_cast<const float2 *>(tops + 2 * r);
                        v[r] = add_f2(x[r], make_float2(-m.x, -m.y));
                    }
                };
                weigh();
                if (cached) {
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) over = max3(over, v[r].x, v[r].y);
                    if (!seen) over = -INFINITY;
                } else {
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) {
                        if (seen >> (2 * r) & 1) over = fmaxf(over, v[r].x);
                        if (seen >> (2 * r + 1) & 1) over = fmaxf(over, v[r].y);
                    }
                }
                if (vote(over > kMost)) {
                    // the rows' maxima over the tile, and m where it has grown
                    float m[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) m[r] = seen >> r & 1 ? (r & 1 ? x[r / 2].y : x[r / 2].x) : -INFINITY;
                    const float mine = over_warp<R, true>(m, lane);
                    if (R == 32 || (lane & 1) == 0) red[warp * R + lane * R / 32] = mine;
                    named_bar_sync(kSoftmaxBar, 128);
                    if (tid < R) {
                        const float was = tops[tid];
                        const float best = fmaxf(fmaxf(red[tid], red[R + tid]), fmaxf(red[2 * R + tid], red[3 * R + tid]));
                        const float now = best == -INFINITY ? was : fmaxf(was, best - kBelow);
                        const bool grows = now > was + kSlack;
                        shrinks[tid] = grows ? ex2(was - now) : 1.f;
                        if (grows) tops[tid] = now;
                    }
                    named_bar_sync(kSoftmaxBar, 128);
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) sum[r] = mul_f2(sum[r], *reinterpret_cast<const float2 *>(shrinks + 2 * r));
                    if (t > w.t0) {
                        // the product of the tile before (the one before that was done with these scores)
                        wait(&bar[B::O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int part = 0; part < pieces; ++part) {
                            uint32_t o[R];
                            tmem_ld<R>(lane_base + COL_O + part * R, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int r = 0; r < R; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * shrinks[r]);
                            if constexpr (R == 16)
                                tmem_st16(lane_base + COL_O + part * R, o);
                            else
                                tmem_st32(lane_base + COL_O + part * R, o);
                        }
                        tmem_st_wait();
                    }
                    weigh();
                }
#pragma unroll
                for (int r = 0; r < R / 2; ++r) {
                    v[r].x = ex2(v[r].x);
                    v[r].y = ex2(v[r].y);
                    if (!cached || !seen) {  // a row's m may still be -inf, a score NaN: what is not seen is 0
                        if (!(seen >> (2 * r) & 1)) v[r].x = 0.f;
                        if (!(seen >> (2 * r + 1) & 1)) v[r].y = 0.f;
                    }
                    sum[r] = fma_f2(v[r], make_float2(inv, inv), sum[r]);
                }
                // where the weights go is free (two places: no faster)
                if (tile > 0) wait(&bar[B::O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
                uint8_t *to = smem + L::kP;
                if (cached) {
#pragma unroll
                    for (int i = 0; i < R / 16; ++i) {
                        uint32_t part[4][kPieces];
#pragma unroll
                        for (int k = 0; k < 4; ++k) pieces4(v[8 * i + 2 * k], v[8 * i + 2 * k + 1], part[k]);
#pragma unroll
                        for (int k = 0; k < kPieces; ++k)
                            *reinterpret_cast<uint4 *>(to + row_offset<kPieces * R>(tid, k * R / 16 + i)) =
                                make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
                    }
                } else {
                    uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
                    for (int i = 0; i < R / 2; ++i) {
                        hi[i] = pack_bf16(v[i].x, v[i].y);
                        lo[i] = pack_bf16((v[i].x - __uint_as_float(hi[i] << 16)) * kUnit,
                                          (v[i].y - __uint_as_float(hi[i] & 0xFFFF0000u)) * kUnit);
                    }
#pragma unroll
                    for (int i = 0; i < R / 8; ++i) {
                        *reinterpret_cast<uint4 *>(to + row_offset<2 * R>(tid, i)) =
                            make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                        *reinterpret_cast<uint4 *>(to + kKeys * 2 * R + row_offset<2 * R>(tid, i)) =
                            make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
                    }
                }
                // the values' row of this thread's key: zeros where there is none, and finite
                const int limit = cached ? w.q.c - base : w.new_seen - base;
                if (!cached || limit < kKeys) {
                    const int i = t - w.t0;
                    const uint32_t pos = ring + stages(min(i + 2, n_tiles)) + stages(i);  // K0 K1 V0 K2 V1 ... V(n-1)
                    const bool second = !cached && kHalves > 1 && tid >= 64;
                    if (!cached && kHalves > 1) wait(&bar[B::KV_FULL0 + (pos + 1) % kRing], ((pos + 1) / kRing) & 1);
                    wait(&bar[B::KV_FULL0 + pos % kRing], (pos / kRing) & 1);
                    uint8_t *tile_at = smem + L::kRing + ((pos + second) % kRing) * kStage;
                    const int row = second ? tid - 64 : tid;
                    if (tid >= limit) {
                        // (the whole of a row: its swizzle does not matter)
                        if (cached) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                reinterpret_cast<uint4 *>(tile_at + row * D)[k] = make_uint4(0, 0, 0, 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < D / 8; ++k)
                                reinterpret_cast<uint4 *>(tile_at + (k >> 3) * 8192 + row * 128)[k & 7] = make_uint4(0, 0, 0, 0);
                        }
                    } else if (!cached) {
#pragma unroll
                        for (int k = 0; k < D / 8; ++k) {
                            uint4 *at = reinterpret_cast<uint4 *>(tile_at + (k >> 3) * 8192 + row * 128) + (k & 7);
                            uint4 u = *at;
                            const uint32_t p0 = nonfinite_bf16x2(u.x), p1 = nonfinite_bf16x2(u.y), p2 = nonfinite_bf16x2(u.z),
                                           p3 = nonfinite_bf16x2(u.w);
                            if (p0 | p1 | p2 | p3) {
                                u.x &= ~p0, u.y &= ~p1, u.z &= ~p2, u.w &= ~p3;
                                *at = u;
                                dirty[item & 1] = item;  // a warp is at most one item ahead of another
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B::P_READY0 + (tile & 1)]);
            }
            ring += 2 * stages(n_tiles);
            // the next item's queries while the last product runs: its first scores need not wait for this one's output
            kvs::Walk next = w;
            more = next.next<true>(a, p.g);
            if (more) split(next, item);
            const bool whole = w.whole();
            const int64_t part = ((int64_t)worker * 2 + (w.t0 > 0 ? 0 : 1)) * p.g.rows;
            // output row of the item's row i: (token0 + i / group, head0 + i mod group)
            const int64_t row0 = (int64_t)(w.q.q0 + token0) * a.nheads + w.h * group;
            auto out_row = [&](int i) {
                return row0 + i + (int64_t)((uint32_t)i * p.group_inv >> 16) * (a.nheads - group);
            };
            {
                float s[R];
#pragma unroll
                for (int r = 0; r < R / 2; ++r) s[2 * r] = sum[r].x, s[2 * r + 1] = sum[r].y;
                const float mine = over_warp<R, false>(s, lane);
                if (R == 32 || (lane & 1) == 0) red[warp * R + lane * R / 32] = mine;
            }
            named_bar_sync(kSoftmaxBar, 128);
            if (tid < R) {
                const float top = tops[tid], total = (red[tid] + red[R + tid]) + (red[2 * R + tid] + red[3 * R + tid]);
                shrinks[tid] = !whole ? 1.f : total == 0.f ? 0.f : 1.f / total;  // a row that saw nothing: zeros
                if (tid < rows) {
                    if (!whole)
                        p.parts.stats[part + tid] = make_float2(top, total);
                    else if (a.lse)
                        a.lse[out_row(tid)] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
                }
            }
            named_bar_sync(kSoftmaxBar, 128);
            wait(&bar[B::O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            float y[R];
#pragma unroll
            for (int r = 0; r < R; ++r) y[r] = 0.f;
#pragma unroll 1
            for (int part = pieces - 1; part >= 0; --part) {  // the smallest first
                uint32_t o[R];
                tmem_ld<R>(lane_base + COL_O + part * R, o);
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < R; ++r) y[r] = fmaf(y[r], 1.f / kUnit, __uint_as_float(o[r]));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) y[r] *= shrinks[r];
            const int d = D == 128 ? tid : tid & 63;  // column
            if (dirty[item & 1] == item) {
                // values that were taken out, to the rows that see them: only decides between infinity and NaN
                for (int j = max(0, w.t0 - w.cached_tiles) * kKeys; j < min(w.new_seen, (w.t1 - w.cached_tiles) * kKeys); ++j) {
                    const float value = to_f32(static_cast<const __nv_bfloat16 *>(a.v_new)[(int64_t)(w.q.q0 + j) * a.v_stride + w.h * D + d]);
                    if (!__any_sync(~0u, !isfinite(value))) continue;
                    const uint32_t seen = seen_by(j);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (!isfinite(value) && (seen >> r & 1)) y[r] += value;
                }
            }
            if (tid < D) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= rows) break;
                    if (whole)
                        static_cast<__nv_bfloat16 *>(a.out)[out_row(r) * D + d] = __float2bfloat16_rn(y[r]);
                    else
                        p.parts.sums[(part + r) * D + d] = y[r];
                }
            }
            w = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

kvs::Tiling few_tiling(const kv_attention_args &a) {
    kvs::Tiling g = kvs::tiling(a, kvs::kFewRows, kKeyShift, kOverhead, 1);
    g.part_cost = 0.05f;  // in tiles of 128 keys
    return g;
}

// CTAs: as many for every key head
int few_workers(const kv_attention_args &a, const kvs::Tiling &g) {
    kv_attention_args one = a;
    one.nheads = a.nheads / a.kv_heads, one.kv_heads = 1;
    const int most = 2 * device_sms() / a.kv_heads;
    return kvs::grid_of(one, g, most < 1 ? 1 : most) * a.kv_heads;
}

template <int D, int R> cudaError_t launch(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    Params p;
    p.a = a;
    p.k_scale = scales.k, p.v_scale = scales.v;
    p.g = few_tiling(a);
    const int workers = few_workers(a, p.g);
    p.parts = kvs::parts_at(ws, workers, p.g.rows, D);
    p.group_inv = (65536u + p.g.heads - 1) / p.g.heads;
    p.box_shift = kKeyShift;
    while (a.block_size % (1 << p.box_shift)) --p.box_shift;
    p.key_shift = 3;  // no more than a request is said to have: decode steps bring few rows
    while (p.key_shift < kKeyShift && (1 << p.key_shift) < a.max_new_tokens) ++p.key_shift;
    p.val_shift = D == 128 && p.key_shift > 6 ? 6 : p.key_shift;
    p.wait_limit = a.wait_limit_cycles > 0 ? a.wait_limit_cycles : 2000000000ll;
    constexpr uint32_t halves = D / 64;
    const uint64_t H = a.nheads, G = a.kv_heads, T = a.total_tokens, rows = a.block_size, blocks = a.num_blocks;
    const uint64_t head = D * 2, k_stride = (uint64_t)a.k_stride * 2, v_stride = (uint64_t)a.v_stride * 2;  // in bytes
    constexpr auto kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap q, kc, vc, kn, vn;
    // caches: a row, rows of a block, heads, blocks; new tokens: 64 columns, tokens, column halves, heads
    const cuuint64_t cache_dims[4] = {D, rows, G, blocks}, cache_strides[3] = {G * D, D, (uint64_t)a.cache_block_stride};
    const cuuint32_t cache_box[4] = {D, 1u << p.box_shift, 1, 1};
    const cuuint64_t new_dims[4] = {64, T, halves, G}, kn_strides[3] = {k_stride, 128, head};
    const cuuint64_t vn_strides[3] = {v_stride, 128, head};
    const cuuint32_t kn_box[4] = {64, 1u << p.key_shift, 1, 1}, vn_box[4] = {64, 1u << p.val_shift, 1, 1};
    const bool ok = make_tmap_bf16_3d(&q, a.q, D, H, T, head, (uint64_t)a.q_stride * 2, 64, p.g.heads, p.g.tokens) &&
                    make_tmap_8bit<4>(&kc, a.k_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_8bit<4>(&vc, a.v_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_16bit<4>(&kn, kType, a.k_new, new_dims, kn_strides, kn_box) &&
                    make_tmap_16bit<4>(&vn, kType, a.v_new, new_dims, vn_strides, vn_box);
    if (!ok) return cudaErrorInvalidValue;
    constexpr int smem = Layout<D, R>::kBytes;
    const auto kernel = kv_attention_fp8_few_kernel<D, R>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<workers, kThreads, smem, s>>>(q, kc, vc, kn, vn, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kvs::join_launch(a, p.parts, workers, p.g, s);
}

template <int D> cudaError_t launch_rows(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    return few_tiling(a).rows <= 16 ? launch<D, 16>(a, scales, ws, s) : launch<D, 32>(a, scales, ws, s);
}

}  // namespace

// Whether tiles of at most 32 rows hold what a request is said to have, or all of a tile of 128: the sizes of the tensor
// cores' kernels are taken for granted.
bool kv_attention_fp8_few(const kv_attention_args &a) {
    const int group = a.nheads / a.kv_heads, tokens = 128 / group, hint = a.max_new_tokens > 0 ? a.max_new_tokens : 1;
    return (hint < tokens ? hint : tokens) * group <= kvs::kFewRows;
}

size_t kv_attention_fp8_few_workspace(const kv_attention_args &a) {
    const kvs::Tiling g = few_tiling(a);
    return kvs::parts_bytes(few_workers(a, g), g.rows, a.headdim);
}

cudaError_t kv_attention_fp8_few_launch(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    return a.headdim == 64 ? launch_rows<64>(a, scales, ws, s) : launch_rows<128>(a, scales, ws, s);
}

}  // namespace ssd
