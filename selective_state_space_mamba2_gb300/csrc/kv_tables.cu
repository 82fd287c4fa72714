// kv_block_tables: block tables, slot map and positions of one step from the requests' lengths.
//
// Everything a token needs follows from three prefix sums over the requests (tokens, blocks
// taken) and its own request's lengths, so one launch does it all: every CTA scans all S
// requests (12 bytes each, from L2 after the first CTA) and then writes only its own tile of
// tokens; no CTA waits for another's result.  A block's table entry is written by the CTA that
// owns the block's first new token.  Requests with many tokens in a tile are queued and
// written by the whole CTA, the others by the thread that scanned them.
// What bounds it: 12 bytes per token at HBM speed in large steps, launch and two dependent
// rounds of loads in small ones.
#include "kv.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 1024;   // tokens of a CTA
constexpr int kInline = 8;    // tokens of a request in a tile that its scanning thread writes itself
constexpr int kQueue = kTile / (kInline + 1) + 2;

struct Span {  // tokens [t0, t1) of request r
    int32_t t0, t1, r, pos0, held, taken;
};

struct Totals {
    unsigned long long tokens, pops;
    uint32_t bad;
};

__device__ __forceinline__ int32_t blocks_of(int32_t tokens, int32_t b) { return tokens / b + (tokens % b != 0); }

struct Lens {
    int32_t c, n, held, need;
    uint32_t bad;
};

__device__ __forceinline__ Lens lens_of(const kv_tables_args &a, int32_t r) {
    Lens l;
    l.c = a.context_lens[r];
    l.n = a.new_lens[r];
    const int32_t v = a.reserved_lens[r];
    l.bad = 0;
    if (l.c < 0 || l.n < 0 || v < 0 || l.c > INT32_MAX - l.n) {
        l.bad = SSD_DEVERR_METADATA;
        l.held = l.need = 0;
        return l;
    }
    l.held = blocks_of(v, a.block_size);
    l.need = max(l.held, blocks_of(l.c + l.n, a.block_size));
    if (l.need > a.table_cols) l.bad = SSD_DEVERR_BLOCKS;
    return l;
}

__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const kv_tables_args a) {
    __shared__ Totals warp_tot[kThreads / 32];
    __shared__ unsigned long long warp_sum[kThreads / 32];
    __shared__ Span queue[kQueue];
    __shared__ int queued;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = a.num_reqs, b = a.block_size;
    if (tid == 0) queued = 0;

    // totals and checks over all requests
    Totals t{0, 0, 0};
    for (int r = tid; r < S; r += kThreads) {
        const Lens l = lens_of(a, r);
        t.bad |= l.bad;
        t.tokens += l.n > 0 ? l.n : 0;
        t.pops += l.need - l.held;
    }
    for (int o = 16; o > 0; o >>= 1) {
        t.tokens += __shfl_xor_sync(~0u, t.tokens, o);
        t.pops += __shfl_xor_sync(~0u, t.pops, o);
        t.bad |= __shfl_xor_sync(~0u, t.bad, o);
    }
    if (lane == 0) warp_tot[warp] = t;
    const int32_t head = a.ring_in[0], count = a.ring_in[1];
    __syncthreads();
    t = Totals{0, 0, 0};
    for (int w = 0; w < kThreads / 32; ++w) {
        t.tokens += warp_tot[w].tokens;
        t.pops += warp_tot[w].pops;
        t.bad |= warp_tot[w].bad;
    }
    if (t.tokens > (unsigned long long)a.max_tokens) t.bad |= SSD_DEVERR_METADATA;
    if (head < 0 || count < 0 || count > a.free_capacity || (head >= a.free_capacity && head > 0))
        t.bad |= SSD_DEVERR_METADATA;
    else if (t.pops > (unsigned long long)count)
        t.bad |= SSD_DEVERR_BLOCKS;
    const bool ok = t.bad == 0;
    if (blockIdx.x == 0 && tid == 0) {
        if (!ok) report(a.err_word, t.bad);
        a.ring_out[0] = ok && t.pops ? (int32_t)((head + t.pops) % a.free_capacity) : head;
        a.ring_out[1] = ok ? count - (int32_t)t.pops : count;
        a.cu_seqlens[S] = ok ? (int32_t)t.tokens : 0;
    }
    const int32_t total = ok ? (int32_t)t.tokens : 0;
    const int32_t tile0 = (int32_t)min((long long)blockIdx.x * kTile, (long long)a.max_tokens);
    const int32_t tile1 = (int32_t)min((long long)tile0 + kTile, (long long)a.max_tokens);

    // padding rows of the tile
    for (int i = max(tile0, total) + tid; i < tile1; i += kThreads) {
        a.slots[i] = -1;
        a.positions[i] = 0;
        if (a.token_req) a.token_req[i] = -1;
    }

    auto token = [&](int32_t i, int32_t r, int32_t pos, int32_t held, int32_t taken, bool first) {
        const int32_t col = pos / b, off = pos - col * b;
        int32_t *row = a.block_table + (int64_t)r * a.table_cols;
        int32_t id;
        if (col < held) {
            id = row[col];
        } else {
            id = a.free_ring[((int64_t)head + taken + (col - held)) % a.free_capacity];
            if (off == 0 || first) row[col] = id;
        }
        int32_t slot = -1;
        if (id != a.null_block_id) {
            if (id < 0 || id >= a.num_blocks)
                report(a.err_word, SSD_DEVERR_SLOT);
            else
                slot = id * b + off;
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
        if (a.token_req) a.token_req[i] = r;
    };

    // prefix sums, 256 requests at a time: tokens in the high half, blocks taken in the low one
    unsigned long long carry = 0;
    for (int base = 0, chunk = 0; base < S; base += kThreads, ++chunk) {
        const int r = base + tid;
        const bool owner = chunk % gridDim.x == blockIdx.x;
        Lens l{0, 0, 0, 0, 0};
        if (r < S && ok) l = lens_of(a, r);
        const unsigned long long own = (unsigned long long)l.n << 32 | (uint32_t)(l.need - l.held);
        unsigned long long sum = own;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += v;
        }
        __syncthreads();  // the last chunk's readers of warp_sum and the queue are done
        if (lane == 31) warp_sum[warp] = sum;
        if (tid == 0) queued = 0;
        __syncthreads();
        unsigned long long before = carry + sum - own;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            carry += warp_sum[w];
        }
        const int32_t first = (int32_t)(before >> 32), taken = (int32_t)(uint32_t)before;
        if (r < S) {
            if (owner) {
                a.cu_seqlens[r] = first;
                const int32_t c = a.context_lens[r], v = a.reserved_lens[r];
                a.seq_lens[r] = ok ? c + l.n : c;
                a.reserved_out[r] = ok ? max(v, c + l.n) : v;
                // new blocks that no new token falls into
                const int32_t last = l.n > 0 ? min(l.need, l.c / b) : l.need;
                for (int col = l.held; col < last; ++col)
                    a.block_table[(int64_t)r * a.table_cols + col] =
                        a.free_ring[((int64_t)head + taken + (col - l.held)) % a.free_capacity];
            }
            const int32_t t0 = max(first, tile0), t1 = min(first + l.n, tile1);
            if (t1 > t0) {
                if (t1 - t0 <= kInline) {
                    for (int i = t0; i < t1; ++i) token(i, r, l.c + (i - first), l.held, taken, i == first);
                } else {
                    queue[atomicAdd(&queued, 1)] = Span{t0, t1, r, l.c + (t0 - first), l.held, taken};
                }
            }
        }
        __syncthreads();
        const int nq = queued;
        for (int q = 0; q < nq; ++q) {
            const Span s = queue[q];
            const int32_t c = a.context_lens[s.r];
            for (int i = s.t0 + tid; i < s.t1; i += kThreads) {
                const int32_t pos = s.pos0 + (i - s.t0);
                token(i, s.r, pos, s.held, s.taken, pos == c);
            }
        }
    }
}

}  // namespace

cudaError_t kv_tables_launch(const kv_tables_args &a, cudaStream_t s) {
    const int64_t grid = ((int64_t)a.max_tokens + kTile - 1) / kTile;
    kv_tables_kernel<<<(unsigned)(grid > 0 ? grid : 1), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ssd
