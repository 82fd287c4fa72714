// How kv_tree_attention's work is cut over the GPU (device code shared by its kernels).
//
// An item is one tile of query rows of one request and key head: `tokens` tokens by the key head's
// query heads, or, where those are more than a tile's rows, one token by `heads` of them (`parts`
// tiles per token).  An item's keys come in tiles of 2^key_shift: first its cached positions, then the request's new
// tokens up to the last one a row of the tile can see.  One (item, key tile) is a unit.  All
// units in order (request, head, row tile, key tile) are cut into as many equal runs as there
// are CTAs, so ragged batches fill the GPU and a long cache is split without the host knowing
// any length.  Each CTA finds its run by scanning the requests' lengths itself.  An item cut by
// a border leaves its parts' unnormalised sums in the workspace; the join kernel adds them up.
#pragma once
#include "kv.cuh"

namespace ssd {
namespace kvs {

// Written by every CTA, for the join kernel: the item that the border before its run cuts.
struct Border {
    int32_t parts;           // 0: the border cuts no item, or is not the first to cut this one; else the
                             // CTAs with a part of it, from the one before the border on
    int32_t token0, tokens;  // rows of the item: first packed token, tokens,
    int32_t head0, heads;    // first query head, query heads
};

// n / d; 64-bit division takes several hundred cycles, and few calls need it.
__device__ __forceinline__ unsigned long long quotient(unsigned long long n, unsigned long long d) {
    return (n | d) >> 32 ? n / d : (uint32_t)n / (uint32_t)d;
}

// Square root, of whatever accuracy; the rounded one's special cases cost the kernels registers all along (trees
// 177 to 183 us).
__device__ __forceinline__ float root(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// `total` units cut into `runs` runs: the first `rem` of them have base + 1, the others base.
struct Cut {
    unsigned long long base, rem;
    __device__ __forceinline__ Cut(unsigned long long total, uint32_t runs) {
        base = quotient(total, runs);
        rem = total - base * runs;
    }
    // first unit of run i
    __device__ __forceinline__ unsigned long long start(uint32_t i) const { return i * base + (i < rem ? i : rem); }
    // the run that unit u is in
    __device__ __forceinline__ uint32_t run_of(unsigned long long u) const {
        const unsigned long long longer = rem * (base + 1);
        return (uint32_t)(u < longer ? quotient(u, base + 1) : rem + quotient(u - longer, base));
    }
};

struct Request {
    int32_t q0, n, c;  // first packed row, new tokens, cached tokens
};

// A request's lengths; one that is inconsistent counts as having no new tokens.
__device__ __forceinline__ Request request(const kv_attention_args &a, int32_t r, bool tell) {
    Request q;
    const int32_t q1 = a.cu_seqlens[r + 1];
    q.q0 = a.cu_seqlens[r];
    q.c = a.context_lens[r];
    q.n = q1 - q.q0;
    if (q.q0 < 0 || q1 < q.q0 || q1 > a.total_tokens || q.c < 0 ||
        (q.n > 0 && ((int64_t)q.c > (int64_t)a.table_cols * a.block_size ||
                     (a.tree_mask && (int64_t)q.n > 32ll * a.mask_words)))) {
        if (tell) report(a.err_word, SSD_DEVERR_METADATA);
        q.n = 0;
    }
    return q;
}

constexpr int kFewRows = 32;  // tiles of at most so many rows are decode's: the join shares their parts over warps

struct Tiling {
    int32_t tokens;     // tokens of a row tile
    int32_t heads;      // query heads of a row tile (the last part of a token may have fewer)
    int32_t parts;      // row tiles side by side over a key head's query heads
    int32_t key_shift;  // key tiles of 2^key_shift
    int32_t overhead;   // units an item counts besides its key tiles
    int32_t rows;       // rows a tile is given in the workspace: tokens * heads
    int32_t min_units;  // a run is at least about that long
    float part_cost;    // what a part costs in the join, in units
};

__host__ __device__ __forceinline__ int32_t ceil_div(int32_t n, int32_t d) { return n / d + (n % d != 0); }

// key tiles of n keys
__device__ __forceinline__ int32_t tiles_of(const Tiling &g, int32_t n) {
    return (int32_t)(((uint32_t)n + (1u << g.key_shift) - 1) >> g.key_shift);
}

// New tokens that the row tiles of token block b can see: those up to its last token, or all with
// a mask.
__device__ __forceinline__ int32_t visible_new(const kv_attention_args &a, const Request &q, const Tiling &g, int32_t b) {
    return a.tree_mask || q.n - b * g.tokens <= g.tokens ? q.n : (b + 1) * g.tokens;
}

// Key tiles that the first `blocks` token blocks of a chain see of its new tokens, none of them the last
// block: sum over b of ceil(b t / K), b = 1 .. blocks, t tokens a block, K keys a tile.  K ceil(x / K) is
// x + (-x mod K), and -b t mod K takes every multiple of K / P below K once in P blocks in a row, P = K / gcd(t, K).
__device__ __forceinline__ long long tiles_before(const Tiling &g, int32_t blocks) {
    const uint32_t t = (uint32_t)g.tokens, mask = (1u << g.key_shift) - 1;
    const int zeros = min(__ffs((int)t) - 1, g.key_shift), p_shift = g.key_shift - zeros;
    const uint32_t b = (uint32_t)blocks, left = b & ((1u << p_shift) - 1);
    unsigned long long rest = (unsigned long long)(b >> p_shift) * ((((1ull << p_shift) - 1) << g.key_shift) / 2);
    uint32_t x = (b - left) * t;  // modulo K is all that counts
    for (uint32_t i = 0; i < left; ++i) {
        x += t;
        rest += (0u - x) & mask;
    }
    return (long long)(((unsigned long long)b * (b + 1) / 2 * t + rest) >> g.key_shift);
}

// Units of one head of a request's first `blocks` token blocks, of all of it with the last.
__device__ __forceinline__ long long units_before(const kv_attention_args &a, const Request &q, const Tiling &g,
                                                  int32_t blocks) {
    const long long fixed = (long long)blocks * (g.overhead + tiles_of(g, q.c));
    const long long fresh = a.tree_mask ? (long long)blocks * tiles_of(g, q.n) : tiles_before(g, blocks);
    return (fixed + fresh) * g.parts;
}
__device__ __forceinline__ long long units_of(const kv_attention_args &a, const Request &q, const Tiling &g) {
    if (q.n <= 0) return 0;
    const int32_t before = ceil_div(q.n, g.tokens) - 1;
    return units_before(a, q, g, before) + (long long)(g.overhead + tiles_of(g, q.c) + tiles_of(g, q.n)) * g.parts;
}

// The items of a CTA's run, one after the other.  Every thread that walks them gets the same
// sequence.
struct Walk {
    Request q;
    int32_t r, h, b, part;  // current item: request, key head, token block, part of its heads
    int32_t blocks;         // token blocks of the request
    int32_t cached_tiles, tiles;  // key tiles: cached ones, and all
    int32_t t0, t1;         // key tiles of the item that fall to this CTA
    int32_t new_seen;       // new tokens the item's keys include
    int32_t used;           // units of the item in the run
    long long left;         // units of the run from the item on

    // The item's part that starts `first` of its units in.
    __device__ __forceinline__ void set_item(const kv_attention_args &a, const Tiling &g, int32_t first) {
        new_seen = visible_new(a, q, g, b);
        cached_tiles = tiles_of(g, q.c);
        tiles = cached_tiles + tiles_of(g, new_seen);
        used = (int32_t)min((long long)(g.overhead + tiles - first), left);
        t0 = max(0, first - g.overhead);
        t1 = first + used - g.overhead;
    }
    __device__ __forceinline__ bool any() const { return t1 > t0; }  // false: the run ends in an item's overhead
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // tokens and query heads of the item
    __device__ __forceinline__ int32_t first_token(const Tiling &g) const { return b * g.tokens; }
    __device__ __forceinline__ int32_t tokens(const Tiling &g) const { return min(g.tokens, q.n - b * g.tokens); }
    __device__ __forceinline__ int32_t heads(const Tiling &g, int32_t group) const {
        return min(g.heads, group - part * g.heads);
    }
    // To the next item; false at the end of the run.
    __device__ __forceinline__ bool next(const kv_attention_args &a, const Tiling &g) {
        left -= used;
        if (left <= 0) return false;
        if (++part == g.parts) {
            part = 0;
            if (++b == blocks) {
                b = 0;
                if (++h == a.kv_heads) {
                    h = 0;
                    do {
                        if (++r >= a.num_seqs) return false;
                        q = request(a, r, false);
                    } while (q.n <= 0);
                    blocks = ceil_div(q.n, g.tokens);
                }
            }
        }
        set_item(a, g, 0);
        return any();
    }
};

struct FindSmem {
    unsigned long long sum[32];
    uint32_t longest[32];
    Walk w;
};

// Called by all threads of the CTA (blockDim.x a multiple of 32): the run of worker `me` of `of` (a CTA,
// or a pair of them that share their runs), or false when it has none.  Latency is all that counts here:
// lengths are read once, S / blockDim.x requests a thread, sums over a prompt's token blocks are closed forms
// (prompts of up to 4096 tokens 5.2 to 3.6 us), and where a run starts is worked out by the one thread that has
// its request.
//
// Shortest run.  An item of L units cut into runs of u takes u + c L / u, with a part's cost c in the join: least at
// u = sqrt(c L).  With runs of 1 / 4 units 2 requests of 20 to 31 tokens over 5419, 8 query heads, take 28.4 /
// 19.4 us (c = 0.4: 5.9), one of 200 tokens 19.0 / 15.3 (min_units), 5 of up to 4 tokens over 2287 16.6 / 13.4
// (c = 0.1: 1.9), but one token over 777 10.5 / 12.7 (1.3).  Where the root says less, a run is one key tile, on
// the CUDA cores (tiles of 32 keys) as on the tensor cores; with runs of two / one there 4 single tokens over up to 274 take
// 12.1 / 10.1 us, 13 of up to 5 over 260 12.4 / 11.2, one over 2000 12.2 / 13.0.
__device__ __forceinline__ bool find_run(const kv_attention_args &a, const Tiling &g, int32_t me, int32_t of,
                                         FindSmem &sm, Border *borders, Walk &w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
    const int S = a.num_seqs;
    const unsigned long long heads = (unsigned long long)a.kv_heads;
    const int per = ceil_div(S, nthr), r0 = tid * per, r1 = (int)min((long long)S, (long long)r0 + per);
    Request q;
    unsigned long long per_head = 0, own = 0;
    q.q0 = q.n = q.c = 0;
    uint32_t longest = 0;
    for (int r = r0; r < r1; ++r) {
        q = request(a, r, blockIdx.x == 0);
        per_head = (unsigned long long)units_of(a, q, g);
        own += per_head * heads;
        if (q.n > 0) longest = max(longest, (uint32_t)(g.overhead + tiles_of(g, q.c) + tiles_of(g, q.n)));
    }
    longest = __reduce_max_sync(~0u, longest);
    unsigned long long sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sm.sum[warp] = sum, sm.longest[warp] = longest;
    __syncthreads();
    unsigned long long before = sum - own, total = 0;
    for (int i = 0; i < nwarp; ++i) {
        const unsigned long long v = sm.sum[i];
        if (i < warp) before += v;
        total += v;
        longest = max(longest, sm.longest[i]);
    }
    const uint32_t shortest = max((uint32_t)root(g.part_cost * (float)longest), (uint32_t)g.min_units);
    // (more units than 32 bits hold are enough for all)
    const uint32_t runs = total >> 31 ? (uint32_t)of : min(((uint32_t)total + shortest - 1) / shortest, (uint32_t)of);
    if ((uint32_t)me >= runs) {
        if (tid == 0) borders[me].parts = 0;
        return false;
    }
    const Cut cut(total, runs);
    const unsigned long long lo = cut.start(me);
    if (before <= lo && lo - before < own) {  // one thread's request
        unsigned long long off = lo - before;
        w.r = r0;
        if (per > 1) {
            for (;; ++w.r) {
                q = request(a, w.r, false);
                per_head = (unsigned long long)units_of(a, q, g);
                if (off < per_head * heads) break;
                off -= per_head * heads;
            }
        }
        w.q = q;
        w.blocks = ceil_div(q.n, g.tokens);
        w.left = (long long)(cut.start(me + 1) - lo);
        w.h = (int32_t)quotient(off, per_head);
        off -= w.h * per_head;
        w.b = 0;
        const int32_t fixed = g.overhead + tiles_of(g, q.c);
        if (a.tree_mask) {
            w.b = (int32_t)quotient(off, (unsigned long long)(fixed + tiles_of(g, q.n)) * g.parts);
        } else if (w.blocks > 1) {
            // units before block b are about parts (b^2 t / 2K + b (fixed + t / 2K + 1/2)): the root, then the last step
            const float half = 0.5f * (float)g.tokens / (float)(1 << g.key_shift), c = (float)fixed + half + 0.5f;
            const float u = (float)off / (float)g.parts;
            w.b = min((int32_t)(2.f * u / (c + root(c * c + 4.f * half * u))), w.blocks - 1);
            while (w.b > 0 && (unsigned long long)units_before(a, q, g, w.b) > off) --w.b;
            while (w.b + 1 < w.blocks && (unsigned long long)units_before(a, q, g, w.b + 1) <= off) ++w.b;
        }
        off -= (unsigned long long)units_before(a, q, g, w.b);
        const int32_t here = fixed + tiles_of(g, visible_new(a, q, g, w.b));  // units of a token block's part
        w.part = g.parts == 1 ? 0 : (int32_t)off / here;
        const int32_t first = (int32_t)off - w.part * here;
        w.set_item(a, g, first);
        sm.w = w;
        Border b;
        const int32_t group = a.nheads / a.kv_heads;
        b.token0 = q.q0 + w.first_token(g);
        b.tokens = w.tokens(g);
        b.heads = w.heads(g, group);
        b.head0 = w.h * group + w.part * g.heads;
        b.parts = 0;
        const unsigned long long tile0 = lo - first + g.overhead;  // unit of the item's first key tile
        if (lo > tile0 && cut.start(me - 1) <= tile0) b.parts = (int32_t)cut.run_of(tile0 + w.tiles - 1) - me + 2;
        borders[me] = b;  // a pair writes the same twice
    }
    __syncthreads();
    w = sm.w;
    return w.any();
}

// ---- workspace: Border [grid], then per CTA two parts (0: the item at the start of the run was
// begun by another CTA; 1: an item begun here and not finished), each sums [rows, D] and
// (maximum, sum) pairs [rows] ----
struct Parts {
    Border *borders;
    float *sums;   // [grid][2][rows][D]
    float2 *stats; // [grid][2][rows]: maximum in the base-2 domain, sum of weights
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

inline size_t parts_bytes(int grid, int rows, int D) {
    return up256(sizeof(Border) * (size_t)grid) + up256((size_t)grid * 2 * rows * D * 4) + up256((size_t)grid * 2 * rows * 8);
}

inline Parts parts_at(void *ws, int grid, int rows, int D) {
    char *p = static_cast<char *>(ws);
    Parts o;
    o.borders = reinterpret_cast<Border *>(p);
    p += up256(sizeof(Border) * (size_t)grid);
    o.sums = reinterpret_cast<float *>(p);
    p += up256((size_t)grid * 2 * rows * D * 4);
    o.stats = reinterpret_cast<float2 *>(p);
    return o;
}

// How a kernel with `rows` rows and 2^key_shift keys to a tile cuts these heads; `side` row tiles are worked on
// side by side.
inline Tiling tiling(const kv_attention_args &a, int rows, int key_shift, int overhead, int side) {
    const int group = a.nheads / a.kv_heads;
    Tiling g;
    g.key_shift = key_shift;
    g.overhead = overhead;
    if (group > rows) {
        g.tokens = 1, g.heads = rows, g.parts = ceil_div(group, rows);
    } else {
        // as many tokens as fit, but no more than a request is said to have, so that decode steps
        // load and join few rows
        g.tokens = rows / group, g.heads = group, g.parts = 1;
        const int hint = a.max_new_tokens > 0 ? a.max_new_tokens : 1;
        if (hint < g.tokens) g.tokens = hint;
    }
    g.tokens *= side;
    g.rows = g.tokens * g.heads;
    g.min_units = g.rows > rows ? 4 : 1;
    g.part_cost = g.rows > kFewRows ? 0.4f : 0.1f;
    return g;
}

// CTAs to launch: `most` at most, fewer where the host's bounds say that there cannot be as many
// units.
inline int grid_of(const kv_attention_args &a, const Tiling &g, int most) {
    const double blocks = (double)a.total_tokens / g.tokens + (a.num_seqs < a.total_tokens ? a.num_seqs : a.total_tokens);
    const double keys = ((double)a.table_cols * a.block_size + a.total_tokens) / (1 << g.key_shift) + 2;
    const double units = blocks * g.parts * (g.overhead + keys) * a.kv_heads / g.min_units;
    return units < (double)most ? (int)(units < 1 ? 1 : units + 1) : most;
}

// Joins the parts of the items that borders cut (one kernel, defined in kv_attention_simt.cu).
cudaError_t join_launch(const kv_attention_args &a, const Parts &p, int grid, const Tiling &g, cudaStream_t s);

}  // namespace kvs
}  // namespace ssd
