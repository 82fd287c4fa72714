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

// First unit of CTA i's run.
__device__ __forceinline__ long long run_start(long long total, int32_t i, int32_t ctas) {
    return (long long)((unsigned long long)total * (unsigned long long)i / (unsigned long long)ctas);
}

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

struct Tiling {
    int32_t tokens;     // tokens of a row tile
    int32_t heads;      // query heads of a row tile (the last part of a token may have fewer)
    int32_t parts;      // row tiles side by side over a key head's query heads
    int32_t key_shift;  // key tiles of 2^key_shift
    int32_t overhead;   // units an item counts besides its key tiles
    int32_t rows;       // rows a tile is given in the workspace: tokens * heads
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

// Units of one head of a request.
__device__ __forceinline__ long long units_of(const kv_attention_args &a, const Request &q, const Tiling &g) {
    if (q.n <= 0) return 0;
    const int32_t blocks = ceil_div(q.n, g.tokens);
    long long sum = (long long)blocks * (g.overhead + tiles_of(g, q.c));
    if (a.tree_mask) {
        sum += (long long)blocks * tiles_of(g, q.n);
    } else {
        for (int32_t b = 0; b < blocks; ++b) sum += tiles_of(g, visible_new(a, q, g, b));
    }
    return sum * g.parts;
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
    long long base, per_head;
    Request q;
    int32_t r;
};

// Called by all threads of the CTA (blockDim.x a multiple of 32): the run of worker `me` of `of` (a CTA,
// or a pair of them that share their runs), or false when it has none.  min_units: a run is at least
// about that long.
__device__ __forceinline__ bool find_run(const kv_attention_args &a, const Tiling &g, int32_t min_units, int32_t me,
                                         int32_t of, FindSmem &sm, Border *borders, Walk &w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
    const int S = a.num_seqs;
    const unsigned long long heads = (unsigned long long)a.kv_heads;
    // units of the requests, a CTA's worth of them at a time, summed over all
    auto scan = [&](int base, bool tell, Request &q, unsigned long long &per_head, unsigned long long &before,
                    unsigned long long &all) {
        const int r = base + tid;
        q.n = 0;
        per_head = 0;
        if (r < S) {
            q = request(a, r, tell);
            per_head = (unsigned long long)units_of(a, q, g);
        }
        const unsigned long long own = per_head * heads;
        unsigned long long sum = own;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += v;
        }
        __syncthreads();
        if (lane == 31) sm.sum[warp] = sum;
        __syncthreads();
        before = sum - own;
        all = 0;
        for (int i = 0; i < nwarp; ++i) {
            if (i < warp) before += sm.sum[i];
            all += sm.sum[i];
        }
    };
    Request q;
    unsigned long long per_head, before, all, total = 0;
    for (int base = 0; base < S; base += nthr) {
        scan(base, blockIdx.x == 0, q, per_head, before, all);
        total += all;
    }
    const unsigned long long most = (total + min_units - 1) / min_units;
    const int ctas = (int)(most < (unsigned)of ? most : (unsigned)of);
    if (me >= ctas) {
        if (tid == 0) borders[me].parts = 0;
        return false;
    }
    const unsigned long long lo = run_start(total, me, ctas), hi = run_start(total, me + 1, ctas);
    unsigned long long carry = 0;
    for (int base = 0; base < S; base += nthr) {
        if (S > nthr) scan(base, false, q, per_head, before, all);  // else the scan above still holds
        if (q.n > 0 && carry + before <= lo && lo - (carry + before) < per_head * heads) {
            sm.r = base + tid;
            sm.q = q;
            sm.base = (long long)(carry + before);
            sm.per_head = (long long)per_head;
        }
        carry += all;
        if (carry > lo) break;
    }
    __syncthreads();

    w.r = sm.r;
    w.q = sm.q;
    w.blocks = ceil_div(w.q.n, g.tokens);
    w.left = (long long)(hi - lo);
    long long off = (long long)lo - sm.base;
    w.h = (int32_t)(off / sm.per_head);
    off -= w.h * sm.per_head;
    w.b = 0;
    const int32_t fixed = g.overhead + tiles_of(g, w.q.c);
    int32_t here;  // units of a token block's part
    if (a.tree_mask) {
        here = fixed + tiles_of(g, w.q.n);
        w.b = (int32_t)(off / ((long long)here * g.parts));
        off -= (long long)w.b * here * g.parts;
    } else {
        while (true) {
            here = fixed + tiles_of(g, visible_new(a, w.q, g, w.b));
            if (off < (long long)here * g.parts) break;
            off -= (long long)here * g.parts;
            ++w.b;
        }
    }
    w.part = g.parts == 1 ? 0 : (int32_t)off / here;
    const int32_t first = (int32_t)off - w.part * here;
    w.set_item(a, g, first);
    if (tid == nthr - 1) {  // not one of the threads that the run starts with
        Border b;
        const int32_t group = a.nheads / a.kv_heads;
        b.token0 = w.q.q0 + w.first_token(g);
        b.tokens = w.tokens(g);
        b.heads = w.heads(g, group);
        b.head0 = w.h * group + w.part * g.heads;
        const long long tile0 = (long long)lo - first + g.overhead;  // unit of the item's first key tile
        b.parts = 0;
        if ((long long)lo > tile0 && run_start((long long)total, me - 1, ctas) <= tile0) {
            // runs differ by one unit at most: the last CTA whose run starts before the item's end
            const long long end = tile0 + w.tiles;
            int last = (int)min((long long)ctas - 1, (long long)((unsigned long long)end * ctas / total) + 1);
            while (run_start((long long)total, last, ctas) >= end) --last;
            b.parts = last - me + 2;
        }
        borders[me] = b;  // a pair writes the same twice
    }
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

// How a kernel with `rows` rows and 2^key_shift keys to a tile cuts these heads.
inline Tiling tiling(const kv_attention_args &a, int rows, int key_shift, int overhead) {
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
    g.rows = g.tokens * g.heads;
    return g;
}

// CTAs to launch: `most` at most, fewer where the host's bounds say that there cannot be as many
// units.
inline int grid_of(const kv_attention_args &a, const Tiling &g, int min_units, int most) {
    const double blocks = (double)a.total_tokens / g.tokens + (a.num_seqs < a.total_tokens ? a.num_seqs : a.total_tokens);
    const double keys = ((double)a.table_cols * a.block_size + a.total_tokens) / (1 << g.key_shift) + 2;
    const double units = blocks * g.parts * (g.overhead + keys) * a.kv_heads / min_units;
    return units < (double)most ? (int)(units < 1 ? 1 : units + 1) : most;
}

// Joins the parts of the items that borders cut (one kernel, defined in kv_attention_simt.cu).
cudaError_t join_launch(const kv_attention_args &a, const Parts &p, int grid, const Tiling &g, cudaStream_t s);

}  // namespace kvs
}  // namespace ssd
