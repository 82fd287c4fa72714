// kv_block_tables: block tables, slot map and positions of one step from the requests' lengths.
//
// Everything a token needs follows from two prefix sums over the requests (tokens, blocks taken)
// and its own request's lengths, so one launch does it all: every CTA scans all S requests (12
// bytes each, from L2 after the first CTA) and then writes only its own tile of tokens; no CTA
// waits for another's result.  A token finds its request by bisection among the 512 just scanned,
// in shared memory.  A block's table entry is written by the thread of the block's first new token.
// What bounds it: 12 bytes per token in large steps (524672 tokens of 392 requests: 6.7 us, of
// which 2 are the launch), two dependent rounds of loads in small ones (256 requests of 4: 4.8 us).
#include "kv.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 2048;   // tokens of a CTA
constexpr int kPer = kTile / kThreads;  // of a thread

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
    // of the chunk's requests: first packed token, context, blocks held, blocks taken before
    __shared__ int32_t first_of[kThreads], context_of[kThreads], held_of[kThreads], taken_of[kThreads];
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
    auto ring_entry = [&](int32_t off) {
        uint32_t i = (uint32_t)head + (uint32_t)off;
        if (i >= (uint32_t)a.free_capacity) i -= (uint32_t)a.free_capacity;
        return a.free_ring + i;
    };
    // block and offset of a position: the high word of a product with floor((2^32 - 1) / b) is the
    // quotient or one less, positions being below 2^31
    const uint32_t inv_b = 0xFFFFFFFFu / (uint32_t)b;
    auto block_of = [&](int32_t p, int32_t &col, int32_t &off) {
        uint32_t q = __umulhi((uint32_t)p, inv_b), r = (uint32_t)p - q * (uint32_t)b;
        if (r >= (uint32_t)b) ++q, r -= (uint32_t)b;
        col = (int32_t)q, off = (int32_t)r;
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
                    a.block_table[(int64_t)r * a.table_cols + col] = *ring_entry(taken + (col - l.held));
            }
        }
        first_of[tid] = first, context_of[tid] = l.c, held_of[tid] = l.held, taken_of[tid] = taken;
        __syncthreads();
        // the chunk's tokens in this tile
        const int32_t from = max(first_of[0], tile0), to = min((int32_t)(ok ? tokens_carry : 0), tile1);
        if (from >= to) continue;
        // The last request that starts at token i or before it: the ones without tokens start where the
        // next does.  No branches: the bisections of a thread's tokens run side by side.
        int at[kPer] = {};
#pragma unroll
        for (int step = kThreads / 2; step > 0; step /= 2)
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (first_of[at[k] + step] <= min(max(tile0 + tid + k * kThreads, from), to - 1)) at[k] += step;
        int32_t pos[kPer], col[kPer], off[kPer], id[kPer];
        bool entry[kPer];  // the first new token of a new block
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int32_t i = min(max(tile0 + tid + k * kThreads, from), to - 1);
            pos[k] = context_of[at[k]] + (i - first_of[at[k]]);
            block_of(pos[k], col[k], off[k]);
            const int32_t fresh = col[k] - held_of[at[k]];
            const int32_t *src = fresh < 0 ? a.block_table + (int64_t)(base + at[k]) * a.table_cols + col[k]
                                           : ring_entry(taken_of[at[k]] + fresh);
            id[k] = *src;
            entry[k] = fresh >= 0 && (off[k] == 0 || i == first_of[at[k]]);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int32_t i = tile0 + tid + k * kThreads;
            if (i < from || i >= to) continue;
            const int32_t req = base + at[k];
            if (entry[k]) a.block_table[(int64_t)req * a.table_cols + col[k]] = id[k];
            int32_t slot = -1;
            if (id[k] != a.null_block_id) {
                if (id[k] < 0 || id[k] >= a.num_blocks)
                    report(a.err_word, SSD_DEVERR_SLOT);
                else
                    slot = id[k] * b + off[k];
            }
            a.slots[i] = slot;
            a.positions[i] = pos[k];
            if (a.token_req) a.token_req[i] = req;
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
