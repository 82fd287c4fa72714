// kv_tree_attention_fp8 on the tensor cores: a cache in 8 bits, tokens in bf16, headdim 64 or 128.
//
// Items, key tiles of 64, roles and barriers are those of kv_attention_tc.cu.  Over cached tiles
//   S = Q K^T          e4m3, K = headdim: the codes as they are; queries as two parts, high and low, each multiplied
//   P = 2^(t - m)      t = s (c / u) ks + log2 vs; one row per thread (TMEM lane), written over S in TMEM as fp16
//   O += P V           fp16, K = 64: the codes of the values widened to fp16, which is exact, in their place in the ring
// with ks, vs the scales of the key's block and u the row's unit: the power of two that puts its largest query entry in
// [128, 256).  A value's scale is part of its weight, and the running maximum m is that of the scaled weights, so blocks of
// any scale share the accumulators; the sum of the weights takes them without (1 / vs, once for the keys of a block).  A weight
// below 2^-126 is lost to both, and with scales of a request at most 2^96 apart it is 2^-41 of the largest or less.  To have scales
// 2^164 apart was measured, for a range that no model's values have: weights made anew for the sum in items with scales
// above 2^20, trees 265 and prompts 1034 to 1076 us for 245 and 980 (few rows 407 to 417 for 392 on the speculative batch, 205 to
// 213 for 184 with 32 rows); weights 2^56 larger until they are rounded, 252 and 1001 (400, 199).
// m is 2^11 below the row's largest when it is set, which may grow by 2^4 before O is rescaled: weights stay below 2^15.
//
// Rounding.  A bf16 query entry has 8 significant bits: the high part takes 4, what is left has 4 more, so both hold it
// but for e4m3's smallest step, 2^-9 u: 2^-17 of the row's largest entry is lost at most.  Weights are rounded to fp16:
// off by 2^-11 of themselves, or 2^-36 of the largest that m was set by.  (With m 2^6 below it fp16's smallest step was 2^-31 of it:
// 65536 equal keys beside one with 0.999 of the weight were off by 2 %, and by 22 % with 0.9999.)  Sums and statistics are fp32.
//
// New tokens are not in the cache: their tiles are bf16, multiplied as in kv_attention_tc.cu with the queries as they were
// given.  A ring stage holds such a tile; a cached one takes half of it, values' codes the second half.
//
// What bounds it: shared memory and the softmax warps that also use it.  A cached tile of 64 keys (D = 128) takes 385 cycles
// of it for the scores (both parts of the queries are read), 128 for the values' product, 128 for the copies and 192 for the
// widening, 833 in all, of 1040 that pass; a tile of the 16-bit kernel 768.  The softmax warps issue 0.46 instructions a
// cycle and scheduler (3 warps a scheduler, each a chain).  Measured on 4 prompts of 512 to 4096 tokens over up to 8192
// (blocks of 64) / 24 trees of 33 to 64 over up to 16384 (blocks of 32): 974 / 245 us (a 16-bit cache: 741 / 188).
// Ways that were measured and not taken, with the time of this one then:
//   constants of every 8 keys, whatever the blocks, not a kernel for each size of their common part   962 / 276 (961 / 240)
//   one loop for cached and new tiles, of twice the code                                            1031 / 295 (962 / 276)
//   eight softmax warps of 96 registers, two threads a row, which vote on the maximum               1114 / 273 (961 / 240)
//   values widened to a place of their own, a ring of 8 KB stages                                   1244 / 306 (1030 / 295)
//   two warps that widen, the softmax in 128 registers / one, in step with the products  1398 / 274, 1481 / 376 (1030 / 295)
//   weights split into two e4m3 parts, values multiplied as they are: two conversions for two weights at half the rate
//   of others                                                                                       1360 / 300 (1168 / 337)
#include <type_traits>

#include "kv_fp8.cuh"
#include "kv_tc.cuh"
#include "tmap.h"

namespace ssd {
namespace {

using namespace tc;
using namespace kvtc;
using fp8::max_u16x2;

constexpr int kThreads = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kOverhead = 3;    // of an item, in key tiles
constexpr int kStages = 5;
constexpr int kScaleRing = 4;   // tiles whose scales are kept: the ring lets keys come three tiles ahead
constexpr float kBelow = 11.f;  // m is so far (base 2) below the largest weight when it is set
constexpr float kSlack = 4.f;   // growth of the largest weight that is let stand: fp16 ends at 2^16

struct Params {
    kv_attention_args a;
    const float *k_scale, *v_scale;
    kvs::Parts parts;
    kvs::Tiling g;
    int32_t pair;         // CTAs that share an item: 1 or 2
    int32_t tile_tokens;  // tokens of a row tile
    uint32_t group_inv;   // ceil(2^16 / query heads per key head): row / group = row * group_inv >> 16, row < 128
    int32_t box_shift;    // rows of a page that one copy brings: a power of two that divides block_size and kKeys
    int32_t new_shift;    // rows of new tokens that one copy brings
    int32_t new_halves;   // 64-column pieces that it brings of them
    long long wait_limit;
};

enum {
    Q_FULL, Q_EMPTY, QP_READY, S_FULL0, S_FULL1, P_READY0, P_READY1,
    O_DONE0, O_DONE1, FIN, SCALES0, KV_FULL0 = SCALES0 + kScaleRing, KV_EMPTY0 = KV_FULL0 + kStages,
    NUM_BARS = KV_EMPTY0 + kStages
};

template <int D> struct Layout {
    static constexpr int kQ = kRows * D * 2;
    // The queries' parts, high, then low, kRows * D bytes each.  D = 128: over the queries (a row's parts are where its
    // halves were), which then come once more for the new tokens.
    static constexpr bool kReload = D == 128;
    static constexpr int kParts = kReload ? 0 : kQ;
    static constexpr int kTile = kKeys * D * 2;                 // a ring stage: a tile of new tokens, or codes in its second half
    static constexpr int kCodes = kTile / 2;                    // where values' codes land: widened in place
    static constexpr int kRing = kParts + kQ;
    static constexpr int kScales = kRing + kStages * kTile;     // [kScaleRing][2][8]: ks, vs of a tile's boxes
    static constexpr int kConsts = kScales + kScaleRing * 64;   // [4 warps][8]: ks, log2 vs, 1 / vs of a tile's boxes
    static constexpr int kBars = kConsts + 4 * 8 * 16;
    static constexpr int kMisc = kBars + NUM_BARS * 8;          // TMEM base, dead mark, items with non-finite values
    static constexpr int kBytes = kMisc + 16;
    static constexpr int kFind = kRing;                         // before the ring is used
    static_assert(kBytes <= 113 * 1024, "two CTAs to an SM");
};

// byte offset of 16-byte piece c of row r in a tile of rows of D bytes
template <int D> __device__ __forceinline__ uint32_t row_offset(uint32_t r, uint32_t c) {
    return D == 128 ? sw128_offset(r, c) : sw64_offset(r, c);
}

// What the scores and weights of a block's keys take: ks, log2 vs, 1 / vs (approximate, and exact for powers of two; an
// error is the same in all the weights of a block: 2^-22 of them)
struct Consts {
    float ks, shift, inv;
    __device__ __forceinline__ Consts(float k, float v) : ks(fmaxf(k, 1e-37f)), shift(log2_of(v)), inv(reciprocal(v)) {}
};

// Takes out of a tile of new tokens' values the rows from `limit` on and values that are not finite.  True if there were
// any of these.  Called by 128 threads.
template <int D> __device__ __forceinline__ bool clean_values(uint8_t *tile, int limit, int tid) {
    constexpr int kPieces = D / 16;  // 16-byte pieces of a thread: two threads per row
    const int row = tid & 63, part = tid >> 6;
    bool found = false;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int piece = part * kPieces + i;  // of the row's D / 8
        uint8_t *p = tile + (piece >> 3) * (kKeys * 128) + sw128_offset(row, piece & 7);
        if (row >= limit) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(0, 0, 0, 0);
        } else {
            uint4 v = *reinterpret_cast<uint4 *>(p);
            const uint32_t x = nonfinite_bf16x2(v.x), y = nonfinite_bf16x2(v.y), z = nonfinite_bf16x2(v.z),
                           w = nonfinite_bf16x2(v.w);
            if (x | y | z | w) {
                found = true;
                v.x &= ~x, v.y &= ~y, v.z &= ~z, v.w &= ~w;
                *reinterpret_cast<uint4 *>(p) = v;
            }
        }
    }
    return found;
}

// The unit that puts magnitudes of up to `top` (bf16 bits, two side by side; they compare as whole numbers, and NaN and
// infinity are larger than any) in [128, 256).
__device__ __forceinline__ float unit_of(uint32_t top2) {
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    const int e = (int)(top >> 7);  // biased exponent
    float unit = __uint_as_float((uint32_t)min(134 + 127 - e, 254) << 23);
    if (e == 255) unit = __uint_as_float(0x7FC00000u);  // the row's scores are NaN
    return top == 0 ? 1.f : unit;
}

// 16 entries (8 words of bf16 pairs) as two e4m3 parts in units of 1 / unit
__device__ __forceinline__ void split16(const uint32_t *x, float unit, uint4 &high, uint4 &low) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = x[2 * i], b = x[2 * i + 1];
        split4(__uint_as_float(a << 16) * unit, __uint_as_float(a & 0xFFFF0000u) * unit, __uint_as_float(b << 16) * unit,
               __uint_as_float(b & 0xFFFF0000u) * unit, hi[i], lo[i]);
    }
    high = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    low = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// Row `row` of the queries as two e4m3 parts; returns 1 / u.
template <int D> __device__ __forceinline__ float split_row(uint8_t *smem, int row) {
    using L = Layout<D>;
    uint32_t x[D / 2], top = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(smem + (c >> 3) * (kRows * 128) + sw128_offset(row, c & 7));
        x[4 * c] = v.x, x[4 * c + 1] = v.y, x[4 * c + 2] = v.z, x[4 * c + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < D / 2; ++i) top = max_u16x2(top, x[i] & 0x7FFF7FFFu);
    const float unit = unit_of(top);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint4 hi, lo;
        split16(x + 8 * c, unit, hi, lo);
        uint8_t *to = smem + L::kParts + row_offset<D>(row, c);
        *reinterpret_cast<uint4 *>(to) = hi;
        *reinterpret_cast<uint4 *>(to + kRows * D) = lo;
    }
    return 1.f / unit;
}

// Four codes as fp16.
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
    uint2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(codes));
    return r;
}

// A tile's values as fp16 (exactly), rows from `limit` on as zeros, where their codes are: a warp has 16 rows, two lanes
// a row, and reads its codes before it writes a value.  With D = 128 a row's values go over its own codes; with 64 over
// those of other warps, too.
template <int D> __device__ __forceinline__ void widen_values(uint8_t *tile, int limit, int warp, int lane) {
    constexpr int kPieces = D / 32;  // of 16 codes, a lane's
    const int row = warp * 16 + (lane >> 1), part = lane & 1;
    uint4 v[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        v[i] = *reinterpret_cast<const uint4 *>(tile + Layout<D>::kCodes + row_offset<D>(row, part * kPieces + i));
    if (D == 64)
        named_bar_sync(1, 128);
    else
        __syncwarp();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (row >= limit) v[i] = make_uint4(0, 0, 0, 0);
        const int c = part * kPieces + i;
        uint8_t *half = tile + (c >> 2) * (kKeys * 128);
        const uint2 x = widen4(v[i].x), y = widen4(v[i].y), z = widen4(v[i].z), u = widen4(v[i].w);
        *reinterpret_cast<uint4 *>(half + sw128_offset(row, (2 * c) & 7)) = make_uint4(x.x, x.y, y.x, y.y);
        *reinterpret_cast<uint4 *>(half + sw128_offset(row, (2 * c + 1) & 7)) = make_uint4(z.x, z.y, u.x, u.y);
    }
}

// kBox: keys of a tile that are all of one block, a power of two from 8 on
template <int D, int kBox> __global__ void __launch_bounds__(kThreads, 2)
    kv_attention_fp8_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKc,
                            const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmKn,
                            const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Layout<D>;
    constexpr int kHalves = D / 64;
    constexpr uint32_t kTmemCols = 256;
    constexpr uint32_t COL_S = 0, COL_O = 128;  // two score tiles of 64 columns, the output
    const kv_attention_args &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int group = a.nheads / a.kv_heads;
    const int rank = blockIdx.x & (p.pair - 1), worker = p.pair > 1 ? blockIdx.x >> 1 : blockIdx.x;
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
        for (int i = 0; i < NUM_BARS; ++i)
            mbar_init(&bar[i], i == P_READY0 || i == P_READY1 || i == QP_READY ? 4 : i >= SCALES0 && i < SCALES0 + kScaleRing ? 8 : 1);
        fence_mbar_init();
        *dead = 0;
        dirty[0] = dirty[1] = 0;
    }
    kvs::Walk w;
    const bool work =
        kvs::find_run(a, p.g, worker, p.pair > 1 ? gridDim.x >> 1 : gridDim.x, *reinterpret_cast<kvs::FindSmem *>(smem + L::kFind),
                      p.parts.borders, w);
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
        uint32_t st = 0, phase = 0;  // ring stage, its phase
        uint32_t items = 0, tile = 0;
        uint32_t asked = 0, asked_q = 0;  // stages and query tiles whose copies were asked for: all up to a wait that gave up
        // A cached tile comes in boxes of rows of one block, 1 to 8 of them: lanes 0 to 7 ask for keys, a box each, and
        // for the box's scales; lanes 8 to 15 for values, one tile behind, as the ring's order is.  (With one set of
        // lanes for both, one after the other, and a scale for every 8 keys, this warp was the bound.)
        struct Page {
            int32_t col, off, id;
        };
        const int my_box = lane & 7, role = lane >> 3;  // 0: keys, 1: values
        const int row0 = my_box << p.box_shift;         // of the tile
        const bool mine = role < 2 && row0 < kKeys;
        const int step = kKeys / a.block_size, step_off = kKeys % a.block_size;
        // This lane's page of cached tile t; its block id is read a tile ahead (kv_attention_tc.cu).
        auto page = [&](int32_t col, int32_t off, int t) {
            Page g{col, off, 0};
            if (t < w.cached_tiles && mine && t * kKeys + row0 < w.q.c) g.id = a.block_table[(int64_t)w.r * a.table_cols + col];
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
        auto stage_after = [&](uint32_t s) { return s + 1 == kStages ? 0 : s + 1; };
        bool gave_up = false;
        // Waits until stage `s` is free; false where a wait gave up, anyone's, now or before: nothing is asked for after that.
        // (A stage counts as free, too, where the products did not wait for its copies, which then are still on their way.)
        auto is_free = [&](uint32_t s, uint32_t parity) {
            if (gave_up) return false;
            wait(&bar[KV_EMPTY0 + s], parity);
            gave_up = __any_sync(~0u, *dead);
            return !gave_up;
        };
        auto boxes_of = [&](int t) { return (min(kKeys, w.q.c - t * kKeys) + (1 << p.box_shift) - 1) >> p.box_shift; };
        // This lane's box of cached tile t into stage s.
        auto ask = [&](uint32_t s, int t, const Page &g) {
            const int boxes = boxes_of(t);
            uint64_t *full = &bar[KV_FULL0 + s];
            if (my_box == 0) mbar_arrive_expect_tx(full, (boxes * D) << p.box_shift);
            if (my_box < boxes) {
                int32_t id = g.id;
                if (id < 0 || id >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    id = a.num_blocks;  // outside the tensor: reads as zeros
                }
                tma_load_4d(smem + L::kRing + s * L::kTile + (role ? L::kCodes : 0) + row0 * D, role ? &tmVc : &tmKc, 0, g.off,
                            w.h, id, full);
            }
        };
        // The next stage for tile t's keys or values alone.
        const int new_per = kHalves / p.new_halves, new_box = lane / new_per, new_half = lane % new_per;
        auto load = [&](bool value, int t, const Page &g) {
            const uint32_t s = st;
            const bool ok = is_free(s, phase ^ 1);
            if ((st = stage_after(st)) == 0) phase ^= 1;
            if (!ok) return;
            ++asked;
            if (t < w.cached_tiles) {
                if (role == (int)value) ask(s, t, g);
            } else {
                const int base = (t - w.cached_tiles) * kKeys;
                const int boxes = (min(kKeys, w.new_seen - base) + (1 << p.new_shift) - 1) >> p.new_shift;
                uint64_t *full = &bar[KV_FULL0 + s];
                if (lane == 0) mbar_arrive_expect_tx(full, (boxes * kHalves * 128) << p.new_shift);
                if (new_box < boxes)
                    tma_load_4d(smem + L::kRing + s * L::kTile + new_half * (kKeys * 128) + (new_box << p.new_shift) * 128,
                                value ? &tmVn : &tmKn, 0, w.q.q0 + base + (new_box << p.new_shift), new_half, w.h, full);
            }
            __syncwarp();
        };
        // Keys of cached tile t and values of the one before it, into the next two stages.
        auto load_both = [&](int t, const Page &g) {
            const uint32_t s0 = st, s1 = stage_after(s0), phase1 = s1 == 0 ? phase ^ 1 : phase;
            st = stage_after(s1);
            const bool ok = is_free(role == 1 ? s1 : s0, (role == 1 ? phase1 : phase) ^ 1);
            phase = st == 0 || s1 == 0 ? phase ^ 1 : phase;
            if (!ok) return;
            asked += 2;
            if (role < 2) ask(role ? s1 : s0, t - role, g);
            __syncwarp();
        };
        // Scales of a cached tile's blocks to their place in shared memory, a pair for each box; each of lanes 0 to 7 arrives on
        // the tile's barrier when its copies are done.  The place is free: a tile's scales are read before its weights
        // are written, and the ring only lets keys come in a few tiles further on.
        auto load_scales = [&](int t, const Page &g) {
            if (gave_up || t >= w.cached_tiles) return;
            if (role == 0) {
                float *to = reinterpret_cast<float *>(smem + L::kScales) + (tile % kScaleRing) * 16 + my_box;
                uint64_t *full = &bar[SCALES0 + tile % kScaleRing];
                if (mine && t * kKeys + row0 < w.q.c && g.id >= 0 && g.id < a.num_blocks) {
                    const int64_t at = (int64_t)g.id * a.kv_heads + w.h;
                    copy4(to, p.k_scale + at);
                    copy4(to + 8, p.v_scale + at);
                    copies_arrive(full);
                } else {
                    to[0] = to[8] = 1.f;
                    mbar_arrive(full);
                }
            }
            ++tile;
            __syncwarp();
        };
        // An item's queries; where their parts are written over them, once more when the scores of the cached tiles are done.
        auto load_queries = [&]() {
            wait(&bar[Q_EMPTY], (items & 1) ^ 1);
            ++items;
            if (!__any_sync(~0u, *dead)) {
                asked_q = items;
                if (lane == 0) mbar_arrive_expect_tx(&bar[Q_FULL], kHalves * p.tile_tokens * group * 128);
                __syncwarp();
                if (lane < kHalves)
                    tma_load_3d(smem + lane * (kRows * 128), &tmQ, lane * 64, w.h * group,
                                w.q.q0 + w.first_token(p.g) + rank * p.tile_tokens, &bar[Q_FULL]);
            }
            __syncwarp();
        };
        bool more = true;
        while (more) {
            Page now = page_of(w.t0);  // of tile t for keys, of tile t - 1 for values (from the second one on)
            load_queries();
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
                    if (L::kReload && t == w.cached_tiles) load_queries();
                }
                load_scales(t, now);
                now = next;
            }
            load(true, w.t1 - 1, now);
            more = w.next(a, p.g);
        }
        // The copies asked for land before the CTA may go, whether a wait gave up before the last was asked for, gives
        // up after it, or none does (then the products have waited for them).
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (uint32_t k = 0; k < kStages && k < asked; ++k)
            mbar_wait(&bar[KV_FULL0 + (asked - 1 - k) % kStages], (asked - 1 - k) / kStages & 1, 20000000ll);
        if (asked_q > 0) mbar_wait(&bar[Q_FULL], (asked_q - 1) & 1, 20000000ll);
    } else if (warp == kMmaWarp) {
        // ---- products --------------------------------------------------------------
        // In the order of kv_attention_tc.cu, and as there: the warp walks along, an elected lane issues from uniform
        // values, and a wait that gave up does not stop it.
        const uint32_t tmu = __shfl_sync(~0u, tm, 0);
        constexpr uint32_t kIdS8 = idesc_e4m3(kRows, kKeys, 0, 0), kIdS = idesc_bf16(kRows, kKeys, 0, 0);
        constexpr uint32_t kIdO16 = idesc_f16(kRows, D, 0, 1), kIdO = idesc_bf16(kRows, D, 0, 1);
        const uint64_t dQ = sw128_desc(smem_u32(smem), 16, 1024);
        const uint64_t dP = D == 128 ? sw128_desc(smem_u32(smem + L::kParts), 16, 1024)
                                     : sw64_desc(smem_u32(smem + L::kParts), 16, 512);
        const uint64_t dK = sw128_desc(smem_u32(smem + L::kRing), 16, 1024);
        const uint64_t dK8 = D == 128 ? dK : sw64_desc(smem_u32(smem + L::kRing), 16, 512);
        const uint64_t dV = sw128_desc(smem_u32(smem + L::kRing), kKeys * 128, 1024);
        uint32_t st = 0, phase = 0;  // ring stage and its phase
        uint32_t tile = 0, items = 0, split = 0;  // split: items whose queries were split
        auto advance = [&]() {
            if (++st == kStages) st = 0, phase ^= 1;
        };
        auto scores = [&](uint32_t g, bool cached, bool last) {  // of tile number g, the last of these queries or not
            wait(&bar[KV_FULL0 + st], phase);
            tc_fence_after();
            const uint32_t sg = __shfl_sync(~0u, st, 0), gg = __shfl_sync(~0u, g, 0);
            const uint32_t d = tmu + COL_S + 64 * (gg & 1);
            if (elect_one()) {
                if (cached) {
                    const uint64_t k0 = desc_at(dK8, sg * L::kTile);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            mma8_ss(d, desc_at(dP, part * kRows * D + 32 * k), desc_at(k0, 32 * k), kIdS8, part + k > 0);
                } else {
                    const uint64_t k0 = desc_at(dK, sg * L::kTile);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(d, desc_at(dQ, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                               desc_at(k0, (k >> 2) * (kKeys * 128) + (k & 3) * 32), kIdS, k > 0);
                }
                mma_commit(&bar[S_FULL0 + (gg & 1)]);
                mma_commit(&bar[KV_EMPTY0 + sg]);
                if (last) mma_commit(&bar[Q_EMPTY]);
            }
            __syncwarp();
            advance();
        };
        auto output = [&](uint32_t g, bool cached, uint32_t add) {  // of tile number g
            wait(&bar[KV_FULL0 + st], phase);
            const uint32_t sg = __shfl_sync(~0u, st, 0), gg = __shfl_sync(~0u, g, 0);
            const uint64_t v0 = desc_at(dV, sg * L::kTile);
            const uint32_t p0 = tmu + COL_S + 64 * (gg & 1), id = cached ? kIdO16 : kIdO;  // weights and values of one type
            wait(&bar[P_READY0 + (g & 1)], (g >> 1) & 1);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k) mma_ts(tmu + COL_O, p0 + 8 * k, desc_at(v0, 2048 * k), id, k > 0 ? 1u : add);
                mma_commit(&bar[O_DONE0 + (gg & 1)]);
                mma_commit(&bar[KV_EMPTY0 + sg]);
            }
            __syncwarp();
            advance();
        };
        bool more = true;
        while (more) {
            const int n = __shfl_sync(~0u, w.t1 - w.t0, 0), cached = __shfl_sync(~0u, w.cached_tiles - w.t0, 0);
            // the scores of the item's tile i: those after which the queries in shared memory may go are the last ones
            auto scores_of = [&](int i) {
                if (i == 0 || (L::kReload && i == cached)) {
                    wait(&bar[Q_FULL], items & 1);
                    ++items;
                }
                scores(tile + i, i < cached, i == n - 1 || (L::kReload && i == cached - 1));
            };
            if (cached > 0) {
                wait(&bar[QP_READY], split & 1);
                ++split;
            }
            scores_of(0);
            for (int i = 1; i < n; ++i) {
                scores_of(i);
                output(tile + i - 1, i - 1 < cached, i > 1);
            }
            output(tile + n - 1, n - 1 < cached, n > 1);
            tile += n;
            more = w.next(a, p.g);
        }
        if (elect_one()) mma_commit(&bar[FIN]);  // everything issued is done before the CTA goes
        mbar_wait(&bar[FIN], 0, 20000000ll);
        __syncwarp();
    } else {
        // ---- softmax and output ------------------------------------------------------
        const float c = a.scale * kLog2e;
        const float *scales = reinterpret_cast<const float *>(smem + L::kScales);
        float4 *consts = reinterpret_cast<float4 *>(smem + L::kConsts) + warp * 8;
        const uint32_t lane_base = tm + ((uint32_t)(warp * 32) << 16);
        uint32_t tile = 0, ring = 0;        // tile number, ring positions used by earlier items
        uint32_t queries = 0, scaled = 0;   // times that queries came, cached tiles
        int item = 0;
        float cu = 0.f;                     // c / u of the row
        // The queries of an item in parts, if it has cached tiles.  The scores of the item before are done.
        auto split = [&](const kvs::Walk &v) {
            const uint32_t came = queries;
            const bool cached = v.t0 < v.cached_tiles;
            queries += L::kReload && cached && v.t1 > v.cached_tiles ? 2 : 1;
            if (!cached) return;
            wait(&bar[Q_FULL], came & 1);
            __syncwarp();
            const int rows = min(p.tile_tokens, v.q.n - v.first_token(p.g) - rank * p.tile_tokens) * group;
            // (rows that are not there are whatever shared memory holds, and only touch their own lanes)
            if (warp * 32 < rows) {
                cu = c * split_row<D>(smem, tid);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[QP_READY]);
        };
        split(w);
        bool more = true;
        while (more) {
            ++item;
            const int token0 = w.first_token(p.g) + rank * p.tile_tokens;
            const int rows = min(p.tile_tokens, w.q.n - token0) * group;  // none or less: an odd row tile's other half
            const bool warp_live = warp * 32 < rows;
            const int tok = tid < rows ? token0 + (int)(tid * p.group_inv >> 16) : -1;
            const int n_tiles = w.t1 - w.t0;
            // Tiles of which some row does not see every key: the last cached one, and new ones from the one of
            // the row tile's first token on.
            const int part_cached = w.q.c % kKeys ? w.cached_tiles - 1 : -1;
            const int part_new = w.cached_tiles + (a.tree_mask ? 0 : (token0 + 1) / kKeys);
            // ring position of the values of the item's tile i: K0 K1 V0 K2 V1 ... V(n-1)
            auto values_at = [&](int i) { return ring + min(i + 1, n_tiles - 1) + i + 1; };
            auto widen = [&](int t) {
                const uint32_t pos = values_at(t - w.t0), at = pos % kStages;
                wait(&bar[KV_FULL0 + at], (pos / kStages) & 1);
                __syncwarp();
                widen_values<D>(smem + L::kRing + at * L::kTile, w.q.c - t * kKeys, warp, lane);
                fence_proxy_async_smem();
            };
            float top = -INFINITY, sum = 0.f;
            // One tile; cached ones and new ones each have a loop of their own, straight code for the most part: with one
            // loop for both the instruction cache was a bound (no instruction for 1.1 cycles an instruction issued, 0.4
            // in the 16-bit kernel).
            auto step = [&](int t, auto is_cached) {
                constexpr bool cached = decltype(is_cached)::value;
                const uint32_t s_col = lane_base + COL_S + 64 * (tile & 1);
                const bool partial = cached ? t == part_cached : t >= part_new;
                const float *sc = scales + (scaled % kScaleRing) * 16;  // ks of the tile's boxes, vs
                if constexpr (cached) {
                    widen(t);
                    if (warp_live) {
                        wait(&bar[SCALES0 + scaled % kScaleRing], scaled / kScaleRing & 1);
                        __syncwarp();
                        if (kBox < kKeys) {
                            if (lane < kKeys / kBox) {
                                const Consts k(sc[lane], sc[8 + lane]);
                                consts[lane] = make_float4(k.ks, k.shift, k.inv, 0.f);
                            }
                            __syncwarp();
                        }
                    }
                    ++scaled;
                }
                wait(&bar[S_FULL0 + (tile & 1)], (tile >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (warp_live) {
                    uint32_t s[64];
                    tmem_ld64(s_col, s);
                    // of the tile: scores in base 2 are s f + shift; its weights count inv times in their sum
                    float f = c, shift = 0.f, inv = 1.f;
                    if (kBox == kKeys && cached) {
                        const Consts k(sc[0], sc[8]);
                        f = fmaxf(cu * k.ks, 1e-37f), shift = k.shift, inv = k.inv;
                    }
                    constexpr bool grouped = kBox < kKeys && cached;
                    tmem_ld_wait();
                    if (__builtin_expect(partial, 0)) {
                        const unsigned long long seen = seen_bits(a, w, t, tok);
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!(seen >> j & 1)) s[j] = 0xFF800000u;  // -inf
                    }
                    auto at = [&](int j) { return __uint_as_float(s[j]); };
                    auto most8 = [&](int j) {
                        return fmaxf(max3(max3(at(j), at(j + 1), at(j + 2)), at(j + 3), at(j + 4)), max3(at(j + 5), at(j + 6), at(j + 7)));
                    };
                    float best = -INFINITY;
                    if constexpr (grouped) {
#pragma unroll
                        for (int g = 0; g < kKeys / kBox; ++g) {
                            const float4 k = consts[g];
                            float m = most8(kBox * g);
#pragma unroll
                            for (int i = 8; i < kBox; i += 8) m = fmaxf(m, most8(kBox * g + i));
                            best = fmaxf(best, fmaf(m, fmaxf(cu * k.x, 1e-37f), k.y));
                        }
                    } else {
                        const float m = max3(most8(0), most8(8), most8(16)), n = max3(most8(24), most8(32), most8(40));
                        best = fmaf(fmaxf(max3(m, most8(48), most8(56)), n), f, shift);
                    }
                    const float now = best == -INFINITY ? top : fmaxf(top, best - kBelow);
                    const bool grows = now > top + kSlack;  // the first seen key too: top is -inf then
                    if (__builtin_expect(t == w.t0, 0)) {
                        top = now;
                    } else if (__builtin_expect(__any_sync(~0u, grows), 0)) {
                        const float shrink = grows ? ex2(top - now) : 1.f;
                        if (grows) top = now;
                        sum *= shrink;
                        // the product of the tile before (the one before that was done with these scores)
                        wait(&bar[O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < D; d += 32) {
                            uint32_t o[32];
                            tmem_ld32(lane_base + COL_O + d, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
                            tmem_st32(lane_base + COL_O + d, o);
                        }
                        tmem_st_wait();
                    }
                    const float from = top == -INFINITY ? 0.f : top;
                    uint32_t pk[32];
                    if constexpr (grouped) {
#pragma unroll
                        for (int g = 0; g < kKeys / kBox; ++g) {
                            const float4 k = consts[g];
                            const float fg = fmaxf(cu * k.x, 1e-37f), m = k.y - from;
                            float2 add = make_float2(0.f, 0.f);
#pragma unroll
                            for (int j = kBox / 2 * g; j < kBox / 2 * (g + 1); ++j) {
                                float2 v = fma_f2(make_float2(at(2 * j), at(2 * j + 1)), make_float2(fg, fg), make_float2(m, m));
                                v.x = ex2(v.x);
                                v.y = ex2(v.y);
                                add = add_f2(add, v);
                                pk[j] = cvt_f16x2(v.x, v.y);
                            }
                            sum = fmaf(add.x + add.y, k.z, sum);
                        }
                    } else {
                        const float2 f2 = make_float2(f, f), m2 = make_float2(shift - from, shift - from);
                        float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float2 v = fma_f2(make_float2(at(2 * j), at(2 * j + 1)), f2, m2);
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            add[j & 1] = add_f2(add[j & 1], v);
                            pk[j] = cached ? cvt_f16x2(v.x, v.y) : pack_bf16(v.x, v.y);
                        }
                        sum = fmaf((add[0].x + add[0].y) + (add[1].x + add[1].y), inv, sum);
                    }
                    tmem_st32(s_col, pk);
                    tmem_st_wait();
                }
                if (!cached && __builtin_expect(partial, 0)) {
                    const uint32_t pos = values_at(t - w.t0), at = pos % kStages;
                    wait(&bar[KV_FULL0 + at], (pos / kStages) & 1);
                    if (clean_values<D>(smem + L::kRing + at * L::kTile, w.new_seen - (t - w.cached_tiles) * kKeys, tid))
                        dirty[item & 1] = item;  // a warp is at most one item ahead of another
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[P_READY0 + (tile & 1)]);
                ++tile;
            };
            int t = w.t0;
            for (; t < min(w.t1, w.cached_tiles); ++t) step(t, std::true_type());
            for (; t < w.t1; ++t) step(t, std::false_type());
            ring += 2 * n_tiles;
            // the next item's queries while the last product runs: its first scores need not wait for this one's output
            kvs::Walk next = w;
            more = next.next(a, p.g);
            if (more) split(next);
            wait(&bar[O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            if (warp_live) {
                // A row's thread writes its 64-byte pieces itself.
                const bool whole = w.whole();
                const bool fix = dirty[item & 1] == item;
                const float mul = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;  // a row that saw nothing: zeros
                const int64_t part = ((int64_t)worker * 2 + (w.t0 > 0 ? 0 : 1)) * p.g.rows + rank * p.tile_tokens * group + tid;
                // output row of the item's row i: (token0 + i / group, head0 + i mod group)
                const int64_t out_row = (int64_t)(w.q.q0 + token0) * a.nheads + w.h * group + tid +
                                        (int64_t)((uint32_t)tid * p.group_inv >> 16) * (a.nheads - group);
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + out_row * D;
                float *sums = p.parts.sums + part * D;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + COL_O + d, o);
                    tmem_ld_wait();
                    if (fix && tok >= 0) {  // on copies: what the call takes by address stays in registers otherwise
                        const kvs::Walk walk = w;
                        uint32_t fixed[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) fixed[j] = o[j];
                        add_nonfinite(a, walk, tok, d, fixed);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fixed[j];
                    }
                    if (tok >= 0 && whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[j + e]) * mul;
                            *reinterpret_cast<uint4 *>(out + d + j) =
                                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                           pack_bf16(v[6], v[7]));
                        }
                    } else if (tok >= 0) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) st_global_32(sums + d + j, o + j);
                    }
                }
                if (tok >= 0) {
                    if (!whole) {
                        p.parts.stats[part] = make_float2(top, sum);
                    } else if (a.lse) {
                        a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                    }
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

kvs::Tiling tc_tiling(const kv_attention_args &a) { return kvs::tiling(a, kRows, kKeyShift, kOverhead, pair_for(a)); }

// workers: CTAs or pairs
int tc_workers(const kv_attention_args &a, const kvs::Tiling &g) {
    return kvs::grid_of(a, g, 2 * device_sms() / pair_for(a));
}

template <int D, int kBox>
cudaError_t launch(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    Params p;
    p.a = a;
    p.k_scale = scales.k, p.v_scale = scales.v;
    p.g = tc_tiling(a);
    p.pair = pair_for(a);
    p.tile_tokens = p.g.tokens / p.pair;
    const int workers = tc_workers(a, p.g);
    p.parts = kvs::parts_at(ws, workers, p.g.rows, D);
    p.group_inv = (65536u + p.g.heads - 1) / p.g.heads;
    p.box_shift = kKeyShift;
    while (a.block_size % (1 << p.box_shift)) --p.box_shift;
    p.new_shift = 3;  // no more than a request is said to have: decode steps bring few rows
    while (p.new_shift < kKeyShift && (1 << p.new_shift) < a.max_new_tokens) ++p.new_shift;
    p.wait_limit = a.wait_limit_cycles > 0 ? a.wait_limit_cycles : 2000000000ll;
    constexpr uint32_t halves = D / 64;
    const uint32_t box = 1u << p.box_shift, fresh = 1u << p.new_shift;
    p.new_halves = fresh == kKeys ? halves : 1;
    const uint64_t H = a.nheads, G = a.kv_heads, T = a.total_tokens, rows = a.block_size, blocks = a.num_blocks;
    const uint64_t head = D * 2, k_stride = (uint64_t)a.k_stride * 2, v_stride = (uint64_t)a.v_stride * 2;  // in bytes
    constexpr auto kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap q, kc, vc, kn, vn;
    // caches: a row, rows of a block, heads, blocks; new tokens: 64 columns, tokens, column halves, heads
    const cuuint64_t cache_dims[4] = {D, rows, G, blocks}, cache_strides[3] = {G * D, D, (uint64_t)a.cache_block_stride};
    const cuuint32_t cache_box[4] = {D, box, 1, 1};
    const cuuint64_t new_dims[4] = {64, T, halves, G}, kn_strides[3] = {k_stride, 128, head};
    const cuuint64_t vn_strides[3] = {v_stride, 128, head};
    const cuuint32_t new_box[4] = {64, fresh, (uint32_t)p.new_halves, 1};
    const bool ok = make_tmap_bf16_3d(&q, a.q, D, H, T, head, (uint64_t)a.q_stride * 2, 64, p.g.heads, p.tile_tokens) &&
                    make_tmap_8bit<4>(&kc, a.k_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_8bit<4>(&vc, a.v_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_16bit<4>(&kn, kType, a.k_new, new_dims, kn_strides, new_box) &&
                    make_tmap_16bit<4>(&vn, kType, a.v_new, new_dims, vn_strides, new_box);
    if (!ok) return cudaErrorInvalidValue;
    constexpr int smem = Layout<D>::kBytes;
    const auto kernel = kv_attention_fp8_kernel<D, kBox>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<workers * p.pair, kThreads, smem, s>>>(q, kc, vc, kn, vn, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kvs::join_launch(a, p.parts, workers, p.g, s);
}

template <int D> cudaError_t launch_dim(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    if (a.block_size % 64 == 0) return launch<D, 64>(a, scales, ws, s);
    if (a.block_size % 32 == 0) return launch<D, 32>(a, scales, ws, s);
    return a.block_size % 16 == 0 ? launch<D, 16>(a, scales, ws, s) : launch<D, 8>(a, scales, ws, s);
}

}  // namespace

size_t kv_attention_fp8_tc_workspace(const kv_attention_args &a) {
    if (kv_attention_fp8_few(a)) return kv_attention_fp8_few_workspace(a);
    const kvs::Tiling g = tc_tiling(a);
    return kvs::parts_bytes(tc_workers(a, g), g.rows, a.headdim);
}

cudaError_t kv_attention_fp8_tc_launch(const kv_attention_args &a, const fp8::Scales &scales, void *ws, cudaStream_t s) {
    if (kv_attention_fp8_few(a)) return kv_attention_fp8_few_launch(a, scales, ws, s);
    return a.headdim == 64 ? launch_dim<64>(a, scales, ws, s) : launch_dim<128>(a, scales, ws, s);
}

}  // namespace ssd
