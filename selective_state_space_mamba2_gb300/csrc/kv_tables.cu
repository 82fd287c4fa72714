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

constexpr int kThreads = 512;
constexpr int kTile = 2048;   // tokens of a CTA
constexpr int kInline = 8;    // tokens of a request in a tile that its scanning thread writes itself
constexpr int kQueue = kTile / (kInline + 1) + 2;

struct Span {  // tokens [t0, t1) of request r
    int32_t t0, t1, r, pos0, held, taken;
    bool begins;  // t0 is the request's first new token
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
    constexpr int kWarps = kThreads / 32;
    __shared__ unsigned long long warp_tokens[kWarps], warp_pops[kWarps];
    __shared__ uint32_t warp_bad[kWarps];
    __shared__ Span queue[kQueue];
    __shared__ int queued;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = a.num_reqs, b = a.block_size;
    const int32_t head = a.ring_in[0], count = a.ring_in[1];

    // One chunk of requests, a thread each: its lengths, the tokens and blocks before it in the chunk
    // and those of the whole chunk.  The sums are 64 bits wide: nothing has been checked yet.
    Lens l;
    unsigned long long tokens_before, pops_before, tokens_all, pops_all;
    uint32_t bad_all;
    auto scan = [&](int base) {
        const int r = base + tid;
        l = Lens{0, 0, 0, 0, 0};
        if (r < S) l = lens_of(a, r);
        const unsigned long long n = l.n > 0 ? l.n : 0, p = l.need - l.held;
        unsigned long long ns = n, ps = p;
        uint32_t bad = l.bad;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long nv = __shfl_up_sync(~0u, ns, o), pv = __shfl_up_sync(~0u, ps, o);
            if (lane >= o) ns += nv, ps += pv;
        }
        bad = __reduce_or_sync(~0u, bad);
        __syncthreads();  // the last chunk's readers are done
        if (lane == 31) warp_tokens[warp] = ns, warp_pops[warp] = ps, warp_bad[warp] = bad;
        if (tid == 0) queued = 0;
        __syncthreads();
        tokens_before = ns - n, pops_before = ps - p;
        tokens_all = pops_all = 0;
        bad_all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) tokens_before += warp_tokens[w], pops_before += warp_pops[w];
            tokens_all += warp_tokens[w], pops_all += warp_pops[w];
            bad_all |= warp_bad[w];
        }
    };

    // totals and checks over all requests
    unsigned long long tokens = 0, pops = 0;
    uint32_t bad = 0;
    for (int base = 0; base < S; base += kThreads) {
        scan(base);
        tokens += tokens_all, pops += pops_all, bad |= bad_all;
    }
    if (tokens > (unsigned long long)a.max_tokens) bad |= SSD_DEVERR_METADATA;
    if (head < 0 || count < 0 || count > a.free_capacity || (head >= a.free_capacity && head > 0))
        bad |= SSD_DEVERR_METADATA;
    else if (pops > (unsigned long long)count)
        bad |= SSD_DEVERR_BLOCKS;
    const bool ok = bad == 0;
    // entry `off` of the ring from its head on; head and off are below its capacity
    auto ring_id = [&](int32_t off) {
        uint32_t i = (uint32_t)head + (uint32_t)off;
        if (i >= (uint32_t)a.free_capacity) i -= (uint32_t)a.free_capacity;
        return a.free_ring[i];
    };
    if (blockIdx.x == 0 && tid == 0) {
        if (!ok) report(a.err_word, bad);
        uint32_t next = (uint32_t)head + (ok ? (uint32_t)pops : 0u);
        if (ok && pops && next >= (uint32_t)a.free_capacity) next -= (uint32_t)a.free_capacity;
        a.ring_out[0] = (int32_t)next;
        a.ring_out[1] = ok ? count - (int32_t)pops : count;
        a.cu_seqlens[S] = ok ? (int32_t)tokens : 0;
    }
    const int32_t total = ok ? (int32_t)tokens : 0;
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
            id = ring_id(taken + (col - held));
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

    unsigned long long tokens_carry = 0, pops_carry = 0;
    for (int base = 0, chunk = 0; base < S; base += kThreads, ++chunk) {
        if (S > kThreads) scan(base);  // else the scan above still holds
        const int r = base + tid;
        // with a refused step every request starts at 0 and has no tokens
        const int32_t n = ok ? l.n : 0;
        const int32_t first = ok ? (int32_t)(tokens_carry + tokens_before) : 0;
        const int32_t taken = ok ? (int32_t)(pops_carry + pops_before) : 0;
        tokens_carry += tokens_all, pops_carry += pops_all;
        if (r < S) {
            if (chunk % gridDim.x == blockIdx.x) {  // the requests' own outputs are dealt out by chunks
                a.cu_seqlens[r] = first;
                const int32_t v = a.reserved_lens[r];
                a.seq_lens[r] = l.c + n;
                a.reserved_out[r] = ok ? max(v, l.c + n) : v;
                // new blocks that no new token falls into
                const int32_t last = !ok ? l.held : n > 0 ? min(l.need, l.c / b) : l.need;
                for (int col = l.held; col < last; ++col)
                    a.block_table[(int64_t)r * a.table_cols + col] = ring_id(taken + (col - l.held));
            }
            const int32_t t0 = max(first, tile0), t1 = min(first + n, tile1);
            if (t1 > t0) {
                if (t1 - t0 <= kInline) {
                    for (int i = t0; i < t1; ++i) token(i, r, l.c + (i - first), l.held, taken, i == first);
                } else {
                    queue[atomicAdd(&queued, 1)] = Span{t0, t1, r, l.c + (t0 - first), l.held, taken, t0 == first};
                }
            }
        }
        __syncthreads();
        const int nq = queued;
        for (int q = 0; q < nq; ++q) {
            const Span s = queue[q];
            for (int i = s.t0 + tid; i < s.t1; i += kThreads)
                token(i, s.r, s.pos0 + (i - s.t0), s.held, s.taken, s.begins && i == s.t0);
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
