// How kv_tree_attention's work is cut over the GPU (device code shared by its kernels).
//
// An item is one tile of query rows of one request and key head: the request's (token, query
// head) rows are numbered token-major, and tile m holds rows [m * row_tile, (m + 1) * row_tile).
// An item's keys come in tiles of key_tile: first its cached positions, then the request's new
// tokens up to the last one a row of the tile can see.  One (item, key tile) is a unit.  All
// units in order (request, head, row tile, key tile) are cut into as many equal runs as there
// are CTAs, so ragged batches fill the GPU and a long cache is split without the host knowing
// any length.  Each CTA finds its run by scanning the requests' lengths itself.  An item cut by
// a border leaves its parts' unnormalised sums in the workspace; the join kernel adds them up.
#pragma once
#include "kv.cuh"

namespace ssd {
namespace kvs {

// Written by a CTA about the item at the start of its run (for the join kernel).
struct Border {
    long long lo;          // first unit of the CTA
    long long item0, item1;  // units of the item that lo falls into
    int32_t r, h, m, ctas; // the item; number of CTAs that have units
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

__device__ __forceinline__ int32_t tiles_of(int32_t n, int32_t tile) { return (n + tile - 1) / tile; }

// New tokens that row tile m can see: those up to its last row's token, or all with a mask.
__device__ __forceinline__ int32_t visible_new(const kv_attention_args &a, const Request &q, int32_t group,
                                               int32_t row_tile, int32_t m) {
    if (a.tree_mask) return q.n;
    const int64_t last = min((int64_t)(m + 1) * row_tile, (int64_t)q.n * group) - 1;
    return (int32_t)(last / group) + 1;
}

__device__ __forceinline__ int32_t row_tiles(const Request &q, int32_t group, int32_t row_tile) {
    return (int32_t)(((int64_t)q.n * group + row_tile - 1) / row_tile);
}

// Units of one head of a request.
__device__ __forceinline__ long long units_of(const kv_attention_args &a, const Request &q, int32_t group,
                                              int32_t row_tile, int32_t key_tile) {
    if (q.n <= 0) return 0;
    const int32_t tiles = row_tiles(q, group, row_tile);
    const long long cached = (long long)tiles * tiles_of(q.c, key_tile);
    if (a.tree_mask) return cached + (long long)tiles * tiles_of(q.n, key_tile);
    long long sum = cached;
    for (int32_t m = 0; m < tiles; ++m) sum += tiles_of(visible_new(a, q, group, row_tile, m), key_tile);
    return sum;
}

// The items of a CTA's run, one after the other.  Every thread that walks them gets the same
// sequence.
struct Walk {
    Request q;
    int32_t r, h, m;        // current item
    int32_t tiles_m;        // row tiles of the request
    int32_t cached_tiles, tiles;  // key tiles: cached ones, and all
    int32_t t0, t1;         // key tiles of the item that fall to this CTA
    int32_t new_seen;       // new tokens the item's keys include
    long long left;         // units of the run from t0 on

    __device__ __forceinline__ void set_item(const kv_attention_args &a, int32_t group, int32_t row_tile,
                                             int32_t key_tile, int32_t first) {
        new_seen = visible_new(a, q, group, row_tile, m);
        cached_tiles = tiles_of(q.c, key_tile);
        tiles = cached_tiles + tiles_of(new_seen, key_tile);
        t0 = first;
        t1 = (int32_t)min((long long)tiles, first + left);
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // To the next item; false at the end of the run.
    __device__ __forceinline__ bool next(const kv_attention_args &a, int32_t group, int32_t row_tile,
                                         int32_t key_tile) {
        left -= t1 - t0;
        if (left <= 0) return false;
        if (++m == tiles_m) {
            m = 0;
            if (++h == a.kv_heads) {
                h = 0;
                do {
                    if (++r >= a.num_seqs) return false;
                    q = request(a, r, false);
                } while (q.n <= 0);
                tiles_m = row_tiles(q, group, row_tile);
            }
        }
        set_item(a, group, row_tile, key_tile, 0);
        return true;
    }
};

struct FindSmem {
    unsigned long long sum[32];
    long long base;
    int32_t r;
};

// Called by all threads of the CTA (blockDim.x a multiple of 32): its run, or false when it has
// none.  min_units: a run is at least that long while there are fewer CTAs' worth of units.
__device__ __forceinline__ bool find_run(const kv_attention_args &a, int32_t group, int32_t row_tile,
                                         int32_t key_tile, int32_t min_units, FindSmem &sm, Border *borders,
                                         Walk &w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
    const int S = a.num_seqs;
    unsigned long long total = 0;
    for (int r = tid; r < S; r += nthr)
        total += (unsigned long long)units_of(a, request(a, r, blockIdx.x == 0), group, row_tile, key_tile);
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    if (lane == 0) sm.sum[warp] = total;
    __syncthreads();
    total = 0;
    for (int i = 0; i < nwarp; ++i) total += sm.sum[i];
    total *= (unsigned long long)a.kv_heads;
    const unsigned long long most = (total + min_units - 1) / min_units;
    const int ctas = (int)(most < gridDim.x ? most : gridDim.x);
    if ((int)blockIdx.x >= ctas) {
        if (blockIdx.x == 0 && tid == 0) borders[0].ctas = 0;
        return false;
    }
    const long long lo = (long long)(total * blockIdx.x / ctas), hi = (long long)(total * (blockIdx.x + 1) / ctas);

    unsigned long long carry = 0;
    for (int base = 0; base < S; base += nthr) {
        const int r = base + tid;
        unsigned long long own = 0;
        if (r < S) own = (unsigned long long)(units_of(a, request(a, r, false), group, row_tile, key_tile) * a.kv_heads);
        unsigned long long sum = own;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += v;
        }
        __syncthreads();
        if (lane == 31) sm.sum[warp] = sum;
        __syncthreads();
        unsigned long long before = carry + sum - own;
        for (int i = 0; i < nwarp; ++i) {
            if (i < warp) before += sm.sum[i];
            carry += sm.sum[i];
        }
        if (own && before <= (unsigned long long)lo && (unsigned long long)lo < before + own) {
            sm.r = r;
            sm.base = (long long)before;
        }
        if (carry > (unsigned long long)lo) break;
    }
    __syncthreads();

    w.r = sm.r;
    w.q = request(a, w.r, false);
    w.tiles_m = row_tiles(w.q, group, row_tile);
    w.left = hi - lo;
    const long long per_head = units_of(a, w.q, group, row_tile, key_tile);
    long long off = lo - sm.base;
    w.h = (int32_t)(off / per_head);
    off -= w.h * per_head;
    w.m = 0;
    const int32_t cached = tiles_of(w.q.c, key_tile);
    while (true) {
        const long long here = cached + tiles_of(visible_new(a, w.q, group, row_tile, w.m), key_tile);
        if (off < here) break;
        off -= here;
        ++w.m;
    }
    w.set_item(a, group, row_tile, key_tile, (int32_t)off);
    if (tid == 0) {
        Border b;
        b.lo = lo;
        b.item0 = lo - off;
        b.item1 = b.item0 + w.tiles;
        b.r = w.r, b.h = w.h, b.m = w.m, b.ctas = ctas;
        borders[blockIdx.x] = b;
    }
    return true;
}

// ---- workspace: Border [grid], then per CTA two parts (0: the item at the start of the run was
// begun by another CTA; 1: an item begun here and not finished), each sums [row_tile, D] and
// (maximum, sum) pairs [row_tile] ----
struct Parts {
    Border *borders;
    float *sums;   // [grid][2][row_tile][D]
    float2 *stats; // [grid][2][row_tile]: maximum in the base-2 domain, sum of weights
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

inline size_t parts_bytes(int grid, int row_tile, int D) {
    return up256(sizeof(Border) * (size_t)grid) + up256((size_t)grid * 2 * row_tile * D * 4) +
           up256((size_t)grid * 2 * row_tile * 8);
}

inline Parts parts_at(void *ws, int grid, int row_tile, int D) {
    char *p = static_cast<char *>(ws);
    Parts o;
    o.borders = reinterpret_cast<Border *>(p);
    p += up256(sizeof(Border) * (size_t)grid);
    o.sums = reinterpret_cast<float *>(p);
    p += up256((size_t)grid * 2 * row_tile * D * 4);
    o.stats = reinterpret_cast<float2 *>(p);
    return o;
}

// Joins the parts of the items that borders cut (one kernel, defined in kv_attention_simt.cu).
cudaError_t join_launch(const kv_attention_args &a, const Parts &p, int grid, int row_tile, cudaStream_t s);

// CTAs to launch: `most` at most, fewer where the host's bounds say that there cannot be as many
// units.
inline int grid_of(const kv_attention_args &a, int row_tile, int key_tile, int min_units, int most) {
    const int64_t group = a.nheads / a.kv_heads;
    const int64_t rows = (int64_t)a.total_tokens * group;
    const int64_t tiles_m = rows / row_tile + (a.num_seqs < a.total_tokens ? a.num_seqs : a.total_tokens);
    const int64_t keys = ((int64_t)a.table_cols * a.block_size + key_tile - 1) / key_tile +
                         ((int64_t)a.total_tokens + key_tile - 1) / key_tile;
    const double units = (double)tiles_m * (double)keys * a.kv_heads / min_units;
    return units < (double)most ? (int)(units < 1 ? 1 : units + 1) : most;
}

}  // namespace kvs
}  // namespace ssd
