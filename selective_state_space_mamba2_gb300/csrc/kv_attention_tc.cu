// kv_tree_attention on the tensor cores: bf16, headdim 64 or 128.
//
// One item (kv_sched.cuh) is up to 128 query rows (tokens x the query heads of one key head)
// against its keys in tiles of 64.  Per tile
//   S = Q K^T          tcgen05, 128 x 64, K = headdim, both K-major from TMA tiles
//   P = exp2(c S - m)  one row per thread (TMEM lane), written over S in TMEM as bf16
//   O += P V           tcgen05, 128 x headdim, K = 64, P from TMEM, V MN-major
// with the running maximum m and the sum of the weights in registers (fp32).  O stays in TMEM; it
// is only rescaled when a row's maximum grows by more than 2^8.  Up to then the weights, at most 2^8,
// and their sum go by the same older m, which cancels but for the rounding of the weights.
// V is bf16, and both operands of a product have one type, so P is, too.  In tiles of at most 32 rows (decode
// steps, short drafts), whose bytes or latency are the bound, it is held in two parts, high and low, side by side
// in the columns that the scores leave, and multiplied by V twice: 2^-15 is lost of a weight instead of 2^-8.  The
// high part is cut off and the low one lifted by 2^-24 of the weight, so that both are above 0 where the weight
// is, and an infinite value gives infinity, not the difference of two.  256 requests of 4 tokens over up to 8192
// 649 us with two parts / 668 with one, one token over 65536 50.1 / 49.4, one over 777 10.8 / 10.3, 16 of 4
// over up to 1000 18.3 / 16.9, 4 single tokens of 64 heads over 4000 17.8 / 16.0.  Tiles of more rows have P rounded
// to bf16, an error of the order of the output's own rounding (0.0018 to 0.0020 of the outputs' norm, 0.0015 without);
// two parts there make 4 prompts 960 to 1000 us from 735 to 755, 24 trees 242 from 186, a tree of 32 tokens over 4000
// 24.3 from 21.9.  The sum of the weights takes them before any rounding.
//
// Roles (192 threads, two CTAs per SM so that one's softmax runs beside the other's products):
// warps 0-3 softmax and output, warp 4 TMA loads, warp 5 the products.  Keys and values pass
// through one ring of 64-row tiles in the order they are used: K0 K1 V0 K2 V1 ...
//
// Requests of more rows than a tile takes (prompts, larger trees) are worked on by pairs of CTAs: an item
// is then two row tiles, one a CTA, and both walk over the same keys at about the same time, so that the
// one that comes second finds them in L2.  Neither waits for the other.
//
// What bounds it.  Few rows a request (decode steps, short drafts): the bytes of the cache, 256 requests
// of 4 tokens over up to 8192 cached 647 to 651 us, 7.0 TB/s.  Prompts and large trees: shared memory.  Of a
// tile's 512 cycles of products S takes 384 instead of 256 (a product 128 x 64 x 16 reads 6 KB), V is
// read in 128, and the copies write 32 KB in 256: 768, and 720 to 790 measured; 4 prompts of 512 to 4096
// tokens over up to 8192 741 to 777 us, 1360 to 1425 TFLOP/s.  Tried against that, and not faster: tiles of 128
// keys with one buffer of scores (the chain of scores, softmax, output then is the bound), two row tiles
// in a CTA, and products of a pair's 256 rows (cta_group::2, half the keys and values in each CTA: 830
// us; the weights of both CTAs have to reach the one that issues, 0.8 us a tile for the chain).
//
// Masked places: a score that must not count is replaced, not added to, so a NaN key is harmless.
// A value enters the product whatever its weight, so in tiles with rows that are not there or
// that some query does not see, the rows that are not there are zeroed in shared memory, and
// values that are not finite are taken out there and added again, to the rows that see them, at
// the end (which then only decides between infinity and NaN).
//
// Waits are bounded: one that gives up marks the CTA, after which no wait of it waits, nothing
// more is issued, and every loop runs to its (finite) end.
#include "kv_sched.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace ssd {
namespace {

using namespace tc;

constexpr int kRows = 128;    // TMEM lanes: query rows of a tile
constexpr int kKeyShift = 6;
constexpr int kKeys = 1 << kKeyShift;  // keys of a tile
constexpr int kThreads = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kStages = 5;
constexpr int kOverhead = 3;  // of an item, in key tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLift = 1.f / (1 << 24);  // see the top
constexpr float kSlack = 8.f;  // growth of a maximum (base 2) that is let stand

struct TcParams {
    kv_attention_args a;
    kvs::Parts parts;
    kvs::Tiling g;
    int32_t tile_tokens;  // tokens of a row tile
    uint32_t group_inv;   // ceil(2^16 / query heads per key head): row / group = row * group_inv >> 16, row < 128
    int32_t box_shift;  // rows of a page that one copy brings: a power of two that divides block_size and kKeys
    int32_t new_shift;  // rows of new tokens that one copy brings, too
    int32_t box_halves, new_halves;  // 64-column pieces that it brings of them
    long long wait_limit;
};

enum { Q_FULL, Q_EMPTY, S_FULL0, S_FULL1, P_READY0, P_READY1, O_DONE0, O_DONE1, FIN, KV_FULL0, KV_EMPTY0 = KV_FULL0 + kStages,
       NUM_BARS = KV_EMPTY0 + kStages };

template <int D> struct Layout {
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kTile = kKeys * D * 2;
    static constexpr int kRing = kQ;
    static constexpr int kBars = kRing + kStages * kTile;
    static constexpr int kMisc = kBars + NUM_BARS * 8;  // TMEM base, dead mark, items with non-finite values
    static constexpr int kFind = (kMisc + 16 + 15) / 16 * 16;
    static constexpr int kBytes = kFind + (int)sizeof(kvs::FindSmem);
};

// A wait that has to wait, or to look at a limit that may be short.
__device__ __noinline__ void wait_long(uint64_t *bar, uint32_t parity, volatile int *dead, uint32_t *err, long long limit) {
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

// Takes out of value tile `tile` what must not be multiplied (see the top): rows from `limit` on,
// and, where `fresh`, non-finite values.  True if there were any.  Called by 128 threads.
template <int D> __device__ __forceinline__ bool clean_values(uint8_t *tile, int limit, bool fresh, int tid) {
    constexpr int kPieces = D / 16;  // 16-byte pieces of a thread: two threads per row
    const int row = tid & 63, part = tid >> 6;
    bool found = false;
    if (row >= limit || fresh) {
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
    }
    return found;
}

// The non-finite values that clean_values took out, added to the 32 output columns from `col` of a
// row that sees their keys.
__device__ __noinline__ void add_nonfinite(const kv_attention_args &a, const kvs::Walk &w, int tok, int col,
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

// kFew: tiles of at most kvs::kFewRows rows, with weights in two parts
template <int D, int kPair, bool kFew>
__global__ void __launch_bounds__(kThreads, 2)
    kv_attention_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKc,
                           const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmKn,
                           const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ TcParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Layout<D>;
    constexpr int kHalves = D / 64;
    constexpr uint32_t kTmemCols = 256;
    constexpr uint32_t COL_S = 0, COL_O = 128;  // two score tiles of 64 columns, the output
    const kv_attention_args &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int group = a.nheads / a.kv_heads;
    const int rank = blockIdx.x % kPair, worker = blockIdx.x / kPair;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *dead = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    volatile int *dirty = reinterpret_cast<volatile int *>(smem + L::kMisc + 8);

    launch_dependents();  // the join kernel may be set up as CTAs of this one end
    // Tensor memory first: the SM only starts its second CTA once the first has given up its right
    // to allocate more (measured: 3.6 us later when it was allocated after find_run).
    if (warp == kMmaWarp) {
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
            mbar_init(&bar[i], i == P_READY0 || i == P_READY1 ? 4 : 1);
        fence_mbar_init();
        *dead = 0;
        dirty[0] = dirty[1] = 0;
    }
    kvs::Walk w;
    const bool work =
        kvs::find_run(a, p.g, worker, gridDim.x / kPair, *reinterpret_cast<kvs::FindSmem *>(smem + L::kFind),
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
        uint32_t st = 0, phase = 0;         // ring stage, its phase
        uint32_t items = 0;
        uint32_t asked = 0, asked_q = 0;    // tiles and query tiles whose copies were asked for: all up to a wait that gave up
        // one copy brings both halves of the columns where it brings all rows
        const int per = kHalves / p.box_halves, my_box = lane / per, my_half = lane % per;
        const int new_per = kHalves / p.new_halves, new_box = lane / new_per, new_half = lane % new_per;
        // This lane's page of cached tile t.  Its block id is only looked at when it is used, so that the read is
        // not waited for before; from tile to tile the page is stepped on (4 prompts of 512 to 4096 tokens 829
        // to 785 us, trees 203 to 191, against two divisions and a wait for the id in every tile).
        struct Page {
            int32_t col, off, id;
        };
        const int step = kKeys / a.block_size, step_off = kKeys % a.block_size;
        auto page = [&](int32_t col, int32_t off, int t) {
            Page g{col, off, 0};
            if (t < w.cached_tiles && my_box < kKeys >> p.box_shift && t * kKeys + (my_box << p.box_shift) < w.q.c)
                g.id = a.block_table[(int64_t)w.r * a.table_cols + col];
            return g;
        };
        auto page_of = [&](int t) {
            const int32_t pos = t * kKeys + (my_box << p.box_shift);
            return page(pos / a.block_size, pos % a.block_size, t);
        };
        auto page_after = [&](const Page &g, int t) {
            const int32_t off = g.off + step_off;
            const bool over = off >= a.block_size;
            return page(g.col + step + over, over ? off - a.block_size : off, t);
        };
        auto load = [&](bool value, int t, Page g) {
            wait(&bar[KV_EMPTY0 + st], phase ^ 1);
            uint8_t *dst = smem + L::kRing + st * L::kTile;
            uint64_t *full = &bar[KV_FULL0 + st];
            if (++st == kStages) st = 0, phase ^= 1;
            if (__any_sync(~0u, *dead)) return;
            ++asked;
            const bool cached = t < w.cached_tiles;
            const int base = (cached ? t : t - w.cached_tiles) * kKeys;
            const int shift = cached ? p.box_shift : p.new_shift;
            const int boxes = (min(kKeys, (cached ? w.q.c : w.new_seen) - base) + (1 << shift) - 1) >> shift;
            if (lane == 0) mbar_arrive_expect_tx(full, (boxes * kHalves * 128) << shift);
            __syncwarp();
            if (cached && my_box < boxes) {
                int32_t id = g.id;
                if (id < 0 || id >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    id = a.num_blocks;  // outside the tensor: reads as zeros
                }
                uint8_t *to = dst + my_half * (kKeys * 128) + (my_box << shift) * 128;
                const CUtensorMap *map = value ? &tmVc : &tmKc;
                tma_load_5d(to, map, 0, g.off, my_half, w.h, id, full);
            } else if (!cached && new_box < boxes) {
                uint8_t *to = dst + new_half * (kKeys * 128) + (new_box << shift) * 128;
                const CUtensorMap *map = value ? &tmVn : &tmKn;
                tma_load_4d(to, map, 0, w.q.q0 + base + (new_box << shift), new_half, w.h, full);
            }
            __syncwarp();
        };
        bool more = true;
        while (more) {
            Page now = page_of(w.t0), before = now;
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
            for (int t = w.t0; t < w.t1; ++t) {
                const Page next = page_after(now, t + 1);  // a tile ahead
                load(false, t, now);
                if (t > w.t0) load(true, t - 1, before);
                before = now;
                now = next;
            }
            load(true, w.t1 - 1, before);
            more = w.next(a, p.g);
        }
        // The copies asked for land before the CTA may go, whether a wait gave up before the last was asked for, gives
        // up after it, or none does (then the products have waited for them).
        for (uint32_t k = 0; k < kStages && k < asked; ++k)
            mbar_wait(&bar[KV_FULL0 + k], (asked - 1 - k) / kStages & 1, 20000000ll);
        if (asked_q > 0) mbar_wait(&bar[Q_FULL], (asked_q - 1) & 1, 20000000ll);
    } else if (warp == kMmaWarp) {
        // ---- products --------------------------------------------------------------
        // The whole warp walks along, one lane issues.  Order: S of tile 0, then for every tile t
        // S of t + 1 and O of t; so the scores of a tile are there when the softmax of the one before
        // is done.  A wait that gave up does not stop this warp: what it then multiplies has no
        // meaning, but is in bounds, and the loops end.
        // What the instructions are issued from is made uniform over the warp (shuffles) and the issuing lane
        // elected, so that descriptors are uniform values: 8 products 128 x 64 x 16 on an SM with busy warps
        // take 56 to 70 cycles each this way, 100 to 200 behind a branch on the lane.
        const uint32_t tmu = __shfl_sync(~0u, tm, 0);
        constexpr uint32_t kIdS = idesc_bf16(kRows, kKeys, 0, 0);
        constexpr uint32_t kIdO = idesc_bf16(kRows, D, 0, 1);
        const uint64_t dQ = sw128_desc(smem_u32(smem), 16, 1024);
        const uint64_t dK = sw128_desc(smem_u32(smem + L::kRing), 16, 1024);
        const uint64_t dV = sw128_desc(smem_u32(smem + L::kRing), kKeys * 128, 1024);
        uint32_t st = 0, phase = 0;  // ring stage and its phase
        uint32_t tile = 0, items = 0;
        auto advance = [&]() {
            if (++st == kStages) st = 0, phase ^= 1;
        };
        auto scores = [&](uint32_t g, bool last) {  // of tile number g, the item's last or not
            wait(&bar[KV_FULL0 + st], phase);
            tc_fence_after();
            const uint32_t sg = __shfl_sync(~0u, st, 0), gg = __shfl_sync(~0u, g, 0);
            const uint64_t k0 = desc_at(dK, sg * L::kTile);
            const uint32_t d = tmu + COL_S + 64 * (gg & 1);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(d, desc_at(dQ, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                           desc_at(k0, (k >> 2) * (kKeys * 128) + (k & 3) * 32), kIdS, k > 0);
                mma_commit(&bar[S_FULL0 + (gg & 1)]);
                mma_commit(&bar[KV_EMPTY0 + sg]);
                if (last) mma_commit(&bar[Q_EMPTY]);
            }
            __syncwarp();
            advance();
        };
        auto output = [&](uint32_t g, uint32_t add) {  // of tile number g
            wait(&bar[KV_FULL0 + st], phase);  // before the weights: most of the time long there
            const uint32_t sg = __shfl_sync(~0u, st, 0), gg = __shfl_sync(~0u, g, 0);
            const uint64_t v0 = desc_at(dV, sg * L::kTile);
            const uint32_t p0 = tmu + COL_S + 64 * (gg & 1);
            wait(&bar[P_READY0 + (g & 1)], (g >> 1) & 1);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(tmu + COL_O, p0 + 8 * k, desc_at(v0, 2048 * k), kIdO, k > 0 ? 1u : add);
                if (kFew) {  // the low parts
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_ts(tmu + COL_O, p0 + 32 + 8 * k, desc_at(v0, 2048 * k), kIdO, 1u);
                }
                mma_commit(&bar[O_DONE0 + (gg & 1)]);
                mma_commit(&bar[KV_EMPTY0 + sg]);
            }
            __syncwarp();
            advance();
        };
        bool more = true;
        while (more) {
            const int n = __shfl_sync(~0u, w.t1 - w.t0, 0);
            wait(&bar[Q_FULL], items & 1);
            ++items;
            scores(tile, n == 1);
            for (int i = 1; i < n; ++i) {
                scores(tile + i, i == n - 1);
                output(tile + i - 1, i > 1);
            }
            output(tile + n - 1, n > 1);
            tile += n;
            more = w.next(a, p.g);
        }
        if (elect_one()) mma_commit(&bar[FIN]);  // everything issued is done before the CTA goes
        mbar_wait(&bar[FIN], 0, 20000000ll);
        __syncwarp();
    } else {
        // ---- softmax and output ------------------------------------------------------
        const float c = a.scale * kLog2e;
        const uint32_t lane_base = tm + ((uint32_t)(warp * 32) << 16);
        uint32_t tile = 0, ring = 0;  // tile number, ring positions used by earlier items
        int item = 0;
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
            float top = -INFINITY, sum = 0.f;
            for (int t = w.t0; t < w.t1; ++t, ++tile) {
                const uint32_t s_col = lane_base + COL_S + 64 * (tile & 1);
                const bool partial = t == part_cached || t >= part_new;
                wait(&bar[S_FULL0 + (tile & 1)], (tile >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                if (warp_live) {
                    uint32_t s[64];
                    tmem_ld64(s_col, s);
                    tmem_ld_wait();
                    if (partial) {
                        const unsigned long long seen = seen_bits(a, w, t, tok);
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!(seen >> j & 1)) s[j] = 0xFF800000u;  // -inf
                    }
                    float b4[4];  // four chains: a single one of 64 would be bound by its latency
#pragma unroll
                    for (int j = 0; j < 4; ++j) b4[j] = __uint_as_float(s[j]);
#pragma unroll
                    for (int j = 4; j < 64; ++j) b4[j & 3] = fmaxf(b4[j & 3], __uint_as_float(s[j]));
                    const float best = fmaxf(fmaxf(b4[0], b4[1]), fmaxf(b4[2], b4[3]));
                    const float now = best == -INFINITY ? top : fmaxf(top, best * c);
                    const bool grows = now > top + kSlack;  // the first seen key too: top is -inf then
                    if (t == w.t0) {
                        top = now;
                    } else if (__any_sync(~0u, grows)) {
                        const float f = grows ? ex2(top - now) : 1.f;
                        if (grows) top = now;
                        sum *= f;
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
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st32(lane_base + COL_O + d, o);
                        }
                        tmem_st_wait();
                    }
                    const float from = top == -INFINITY ? 0.f : top;
                    const float2 c2 = make_float2(c, c), m2 = make_float2(-from, -from);
                    float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t pk[32], lo[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float2 v = make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                        v = fma_f2(v, c2, m2);
                        v.x = ex2(v.x);
                        v.y = ex2(v.y);
                        add[j & 1] = add_f2(add[j & 1], v);
                        if (kFew) {
                            const uint32_t x = __float_as_uint(v.x), y = __float_as_uint(v.y);
                            pk[j] = __byte_perm(x, y, 0x7632);
                            const float2 high = make_float2(__uint_as_float(x & 0xFFFF0000u), __uint_as_float(y & 0xFFFF0000u));
                            const float2 rest = fma_f2(high, make_float2(-1.f, -1.f), v);
                            v = fma_f2(v, make_float2(kLift, kLift), rest);
                            lo[j] = pack_bf16(v.x, v.y);
                        } else {
                            pk[j] = pack_bf16(v.x, v.y);
                        }
                    }
                    sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
                    tmem_st32(s_col, pk);
                    if (kFew) tmem_st32(s_col + 32, lo);
                    tmem_st_wait();
                }
                if (partial) {
                    const bool cached = t < w.cached_tiles;
                    const int limit = cached ? w.q.c - t * kKeys : w.new_seen - (t - w.cached_tiles) * kKeys;  // rows there
                    // ring position of this tile's values: K0 K1 V0 K2 V1 ... V(n-1)
                    const int i = t - w.t0;
                    const uint32_t pos = ring + (i == n_tiles - 1 ? 2 * n_tiles - 1 : 2 * i + 2);
                    wait(&bar[KV_FULL0 + pos % kStages], (pos / kStages) & 1);
                    if (clean_values<D>(smem + L::kRing + (pos % kStages) * L::kTile, limit, !cached, tid))
                        dirty[item & 1] = item;  // a warp is at most one item ahead of another
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[P_READY0 + (tile & 1)]);
            }
            ring += 2 * n_tiles;
            wait(&bar[O_DONE0 + ((tile - 1) & 1)], ((tile - 1) >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            if (warp_live) {
                // A row's thread writes its 64-byte pieces itself: a query tile is free for the next
                // item's queries as soon as its last scores are done, not after this.
                const bool whole = w.whole();
                const bool fix = dirty[item & 1] == item;
                const float mul = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;  // a row that saw nothing: zeros
                const int64_t part = ((int64_t)worker * 2 + (w.t0 > 0 ? 0 : 1)) * p.g.rows + rank * p.tile_tokens * group +
                                     warp * 32;
                // output row of the item's row i: (token0 + i / group, head0 + i mod group)
                const int64_t row0 = (int64_t)(w.q.q0 + token0) * a.nheads + w.h * group;
                auto out_row = [&](int i) {
                    const int k = (int)((uint32_t)i * p.group_inv >> 16);
                    return row0 + (int64_t)k * (a.nheads - group) + i;
                };
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + out_row(tid) * D;
                float *sums = p.parts.sums + (part + lane) * D;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + COL_O + d, o);
                    tmem_ld_wait();
                    if (fix && tok >= 0) {  // on copies: what the call takes by address stays in registers otherwise
                        const kvs::Walk at = w;
                        uint32_t fixed[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) fixed[j] = o[j];
                        add_nonfinite(a, at, tok, d, fixed);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fixed[j];
                    }
                    if (tok >= 0 && whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[j + e]) * mul;
                            *reinterpret_cast<uint4 *>(out + d + j) =
                                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                           pack_bf16(f[6], f[7]));
                        }
                    } else if (tok >= 0) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) st_global_32(sums + d + j, o + j);  // whole sectors: trees 188 to 184 us
                    }
                }
                if (tok >= 0) {
                    if (!whole) {
                        p.parts.stats[part + lane] = make_float2(top, sum);
                    } else if (a.lse) {
                        a.lse[out_row(tid)] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
                    }
                }
            }
            more = w.next(a, p.g);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

// CTAs that share an item, by a rule on sizes: a pair where the requests have more rows than a tile
// takes on the average, and its two row tiles see the same keys but for one tile of them at most: with a
// mask, or where they are 64 tokens or fewer.  Measured alone / in pairs: 4 prompts of 512 to 4096 tokens
// over up to 8192 cached, 4 query heads to a key head, 771 / 747 to 777 us; 24 trees of 33 to 64 tokens over up
// to 16384, 8 query heads, 209 / 184 to 188 us, of 33 to 48 with 4 heads 297 / 184; 2 times 512 tokens over 65536
// 553 / 444; 64 requests of 1 to 600 over up to 8192 1632 / 1210; but a prompt of 512 tokens beside 64 single
// tokens 187 / 221, since one CTA of the pair then has no rows most of the time.
int pair_for(const kv_attention_args &a) {
    const int64_t group = a.nheads / a.kv_heads;
    const bool many = (int64_t)a.total_tokens * group > (int64_t)kRows * a.num_seqs;
    return many && (a.mask_words > 0 || 2 * (kRows / group) <= kKeys) ? 2 : 1;
}

kvs::Tiling tc_tiling(const kv_attention_args &a) { return kvs::tiling(a, kRows, kKeyShift, kOverhead, pair_for(a)); }

// workers: CTAs or pairs
int tc_workers(const kv_attention_args &a, const kvs::Tiling &g) {
    return kvs::grid_of(a, g, 2 * device_sms() / pair_for(a));
}

template <int D, int kPair, bool kFew> cudaError_t launch(const kv_attention_args &a, void *ws, cudaStream_t s) {
    TcParams p;
    p.a = a;
    p.g = tc_tiling(a);
    p.tile_tokens = p.g.tokens / kPair;
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
    p.box_halves = box == kKeys ? halves : 1;
    p.new_halves = fresh == kKeys ? halves : 1;
    const uint64_t H = a.nheads, G = a.kv_heads, T = a.total_tokens, rows = a.block_size, blocks = a.num_blocks;
    const uint64_t head = D * 2, line = G * head, block = (uint64_t)a.cache_block_stride * 2;  // strides in bytes
    const uint64_t k_stride = (uint64_t)a.k_stride * 2, v_stride = (uint64_t)a.v_stride * 2;
    constexpr auto kType = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap q, kc, vc, kn, vn;
    // caches: 64 columns, rows of a block, column halves, heads, blocks; new tokens the same without blocks
    const cuuint64_t cache_dims[5] = {64, rows, halves, G, blocks}, cache_strides[4] = {line, 128, head, block};
    const cuuint32_t cache_box[5] = {64, box, (uint32_t)p.box_halves, 1, 1};
    const cuuint64_t new_dims[4] = {64, T, halves, G}, kn_strides[3] = {k_stride, 128, head};
    const cuuint64_t vn_strides[3] = {v_stride, 128, head};
    const cuuint32_t new_box[4] = {64, fresh, (uint32_t)p.new_halves, 1};
    const bool ok = make_tmap_bf16_3d(&q, a.q, D, H, T, head, (uint64_t)a.q_stride * 2, 64, p.g.heads, p.tile_tokens) &&
                    make_tmap_16bit<5>(&kc, kType, a.k_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_16bit<5>(&vc, kType, a.v_cache, cache_dims, cache_strides, cache_box) &&
                    make_tmap_16bit<4>(&kn, kType, a.k_new, new_dims, kn_strides, new_box) &&
                    make_tmap_16bit<4>(&vn, kType, a.v_new, new_dims, vn_strides, new_box);
    if (!ok) return cudaErrorInvalidValue;
    constexpr int smem = Layout<D>::kBytes;
    const auto kernel = kv_attention_tc_kernel<D, kPair, kFew>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<workers * kPair, kThreads, smem, s>>>(q, kc, vc, kn, vn, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kvs::join_launch(a, p.parts, workers, p.g, s);
}

template <int D> cudaError_t launch_dim(const kv_attention_args &a, void *ws, cudaStream_t s) {
    if (pair_for(a) > 1) return launch<D, 2, false>(a, ws, s);
    return tc_tiling(a).rows <= kvs::kFewRows ? launch<D, 1, true>(a, ws, s) : launch<D, 1, false>(a, ws, s);
}

}  // namespace

// A rule on sizes alone: what the TMA boxes and the two products take.  A negative scale would
// turn the maximum of the scores into that of their opposites, and zero times the minus infinity
// that stands for a masked score is NaN.
bool kv_attention_tc_supported(const kv_attention_args &a) {
    return a.dtype == SSD_BF16 && (a.headdim == 64 || a.headdim == 128) && a.nheads / a.kv_heads <= kRows &&
           a.block_size % 8 == 0 && a.scale > 0.f && a.cache_block_stride < (int64_t{1} << 38) &&
           a.q_stride < (int64_t{1} << 38) && a.k_stride < (int64_t{1} << 38) && a.v_stride < (int64_t{1} << 38);
}

size_t kv_attention_tc_workspace(const kv_attention_args &a) {
    const kvs::Tiling g = tc_tiling(a);
    return kvs::parts_bytes(tc_workers(a, g), g.rows, a.headdim);
}

cudaError_t kv_attention_tc_launch(const kv_attention_args &a, void *ws, cudaStream_t s) {
    return a.headdim == 64 ? launch_dim<64>(a, ws, s) : launch_dim<128>(a, ws, s);
}

}  // namespace ssd
