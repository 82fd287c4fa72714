// kv_verify_tokens: which drafted tokens stand, and the token that follows them.
//
// A request is worked on by a cluster of 1 to 8 CTAs, each with an equal stretch of the vocabulary.  The walk down
// the tree needs few numbers, so every CTA makes it for itself (its first warp, 32 tokens at a time, all that
// they need loaded at once); a sum over the vocabulary is what costs: once at the end, and once for each drawn
// token that is turned down in a tree.  Weights are whole multiples of 2^-44 in 64 bits, so that sums are exact, the
// same in any order, and every CTA decides alike.  The row is summed in segments of 1024 entries, whose sums stay
// in shared memory: the one that the drawn mark falls into is read again and walked through.
// Bound by the bytes of the rows (256 chains of 1 + 3 over 65536 fp32 entries, 134 MB, 25 to 27 us, 0.73 to 0.8 of the copy
// rate; again on the same rows, of which L2 holds a part, 19.8), or by latency for a few requests (5 trees of 24 over 50021
// entries 10 to 12 us, again on the same rows 8.6: the walk by one warp, then the sum; 12.0 with the drafted
// tokens read again where they are needed and the mark's segment walked through by one warp, and the chains 23.5).
#include <cooperative_groups.h>

#include "kv_fp8.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 1024;                 // entries
constexpr int kMostSegments = (1 << 18) / kSegment + 2;
constexpr int kMostCluster = 8;
constexpr int kKept = 256;                     // tokens of a request whose parents, ids and probabilities stay in shared memory
constexpr double kUnit = 17592186044416.;      // 2^44

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float positive(float v) { return v > 0.f ? v : 0.f; }  // of NaN: 0

// max(p - c q, 0), product and difference rounded one after the other
__device__ __forceinline__ float rest_of(float p, float q, float c) {
    return positive(__fsub_rn(positive(p), __fmul_rn(c, positive(q))));
}

// floor(2^44 x) of an x in [0, 1], as 2^22 high + low.  Sums towards 0 with 2 leave the first 22 places in the mantissa, what
// they cut off is exact, and has the next 22: additions only (a conversion to 64 bits runs at a fraction of their rate).
// Both parts come with `kBias` on them, and are summed as they are.
constexpr uint32_t kBias = 0x40000000u;  // the bits of 2
struct Fixed {
    uint32_t high, low;
    __device__ __forceinline__ explicit Fixed(float x) {
        const float t = __fadd_rz(x, 2.f);
        high = __float_as_uint(t);
        low = __float_as_uint(__fmaf_rz(__fsub_rn(x, __fsub_rn(t, 2.f)), 4194304.f, 2.f));
    }
};
// The sum of n of them (n 2^22 fits 32 bits), high and low parts added up.
__device__ __forceinline__ u64 fixed_sum(uint32_t high, uint32_t low, uint32_t n) {
    return ((u64)(high - n * kBias) << 22) + (low - n * kBias);
}

// The weight of max(p - c q, 0), at most 1, as a whole number of 2^-44; of NaN 0
__device__ __forceinline__ float capped(float p, float q, float c) {
    float r;
    asm("sub.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(p), "f"(__fmul_rn(c, positive(q))));
    return r;
}
__device__ __forceinline__ float capped(float p) { return __saturatef(p); }
__device__ __forceinline__ u64 weight_of(float x) {
    const Fixed f(x);
    return fixed_sum(f.high, f.low, 1);
}

__device__ __forceinline__ void unpack(uint4 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

struct Shared {
    u64 segment[kMostSegments];
    u64 totals[2][kMostCluster];  // every CTA's own sum, written here by that CTA
    u64 all, before;              // the row's sum, that of the CTAs before this one
    u64 steps[kWarps], rest;      // of the segment that the mark falls into: sums of its steps, what is left of the mark
    uint32_t turned_down[kSegment / 32];
    int32_t up[kKept], tok[kKept];  // a token's parent (-1: none that counts), its id
    float p[kKept];                 // and what the target gives it behind its parent
    int32_t cur, count, found;    // walk's end: last token, number of tokens; the segment
    float c;
    double left;
    bool more;                    // the walk waits for a sum
    bool tried;                   // the children of cur were tried
};

// One row of probabilities (and the draft's beside it) as this CTA sees it.
template <typename T> struct Row {
    const T *p, *q;  // q may be null
    float c;
    int V, shift;    // entries before the row since the last 16-byte boundary
    bool together;   // q has the same boundaries

    __device__ Row(const kv_verify_args &a, int64_t row, float c_, bool with_q) {
        p = static_cast<const T *>(a.target_probs) + row * a.target_stride;
        q = with_q ? static_cast<const T *>(a.draft_probs) + row * a.draft_stride : nullptr;
        c = c_, V = a.vocab;
        shift = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
        together = q && (reinterpret_cast<uintptr_t>(q) & 15u) == (reinterpret_cast<uintptr_t>(p) & 15u);
    }
    __device__ int segments() const { return (V + shift + kSegment - 1) / kSegment; }
    __device__ __forceinline__ int segment_of(int v) const { return (v + shift) / kSegment; }
    __device__ __forceinline__ float at(int v) const { return q ? capped(to_f32(p[v]), to_f32(q[v]), c) : capped(to_f32(p[v])); }
    // the kVec entries from v on (v + shift a multiple of kVec; those outside the row are 0)
    __device__ __forceinline__ void get(int v, float (&rest)[kVec<T>]) const {
        constexpr int N = kVec<T>;
        if (v < 0 || v + N > V) {
#pragma unroll
            for (int i = 0; i < N; ++i) rest[i] = v + i >= 0 && v + i < V ? at(v + i) : 0.f;
            return;
        }
        float x[N], y[N];
        unpack(__ldg(reinterpret_cast<const uint4 *>(p + v)), x);
        if (together) {
            unpack(__ldg(reinterpret_cast<const uint4 *>(q + v)), y);
        } else if (q) {
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = to_f32(q[v + i]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) rest[i] = q ? capped(x[i], y[i], c) : capped(x[i]);
    }
};

// Sum of the weights of segment g of a row, by one warp.  A segment inside the row is read kBatch steps at a time, all
// loads before the first use.
template <typename T> __device__ __forceinline__ u64 segment_sum(const Row<T> &row, int g) {
    constexpr int N = kVec<T>, kSteps = kSegment / (32 * N), kBatch = 4;
    const int first = g * kSegment - row.shift, v0 = first + (threadIdx.x & 31) * N;
    uint32_t high = 0, low = 0;
    if (first >= 0 && first + kSegment <= row.V && (row.together || !row.q)) {
#pragma unroll 1
        for (int i = 0; i < kSteps; i += kBatch) {
            uint4 p[kBatch], q[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                p[k] = __ldg(reinterpret_cast<const uint4 *>(row.p + v0 + (i + k) * 32 * N));
                if (row.q) q[k] = __ldg(reinterpret_cast<const uint4 *>(row.q + v0 + (i + k) * 32 * N));
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float x[N], y[N];
                unpack(p[k], x);
                if (row.q) unpack(q[k], y);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const Fixed f(row.q ? capped(x[e], y[e], row.c) : capped(x[e]));
                    high += f.high, low += f.low;
                }
            }
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < kSteps; ++i) {
            float rest[N];
            row.get(v0 + i * 32 * N, rest);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const Fixed f(rest[e]);
                high += f.high, low += f.low;
            }
        }
    }
    u64 sum = fixed_sum(high, low, kSegment / 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return sum;
}

template <typename T> __global__ void __launch_bounds__(kThreads, 4) kv_verify_kernel(const kv_verify_args a, const int ctas) {
    __shared__ Shared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % ctas, r = blockIdx.x / ctas;
    const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1];
    const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_tokens;
    const int n = bad ? 0 : q1 - q0;
    int32_t *path = a.path + (int64_t)r * a.max_path;
    if (n == 0) {  // the whole cluster
        if (rank == 0) {
            for (int i = tid; i < a.max_path; i += kThreads) path[i] = -1;
            if (tid == 0) {
                a.path_lens[r] = 0, a.accepted[r] = 0, a.next_tokens[r] = -1;
                if (bad) report(a.err_word, SSD_DEVERR_METADATA);
            }
        }
        return;
    }
    // The other CTAs' shared memory is only written to once they are known to run: waited for before the first sum.
    if (ctas > 1) cg::this_cluster().barrier_arrive();
    const float draw = a.uniform[q0];  // of the next token
    uint32_t round = 0;

    // Sums of row's weights: s.segment (this CTA's), s.before, s.all.  `drop`: tokens that were turned down at
    // `cur` weigh nothing.  Called by all threads of the cluster; nothing is written to another CTA's shared memory
    // after the last call's barrier, so a CTA may go when it is done.
    const bool kept = n <= kKept;
    // Whether token j was tried behind `cur`, and is x (x < 0: anything)
    auto tried = [&](int j, int cur, int32_t x) {
        const int32_t up = kept ? s.up[j] : a.parents ? a.parents[q0 + j] : j - 1;
        return up == cur && (x < 0 || (kept ? s.tok[j] : a.tokens[q0 + j]) == x);
    };
    auto first_segment = [&](const Row<T> &row, int k) { return (int)((int64_t)row.segments() * k / ctas); };
    auto sum_row = [&](const Row<T> &row, bool drop, int cur) {
        const int g0 = first_segment(row, rank), g1 = first_segment(row, rank + 1);
        for (int g = g0 + warp; g < g1; g += kWarps) {
            const u64 sum = segment_sum(row, g);
            if (lane == 0) s.segment[g - g0] = sum;
        }
        if (ctas > 1 && round == 0) cg::this_cluster().barrier_wait();
        __syncthreads();
        if (drop) {
            for (int j = cur + 1 + tid; j < n; j += kThreads) {
                if (!tried(j, cur, -1)) continue;
                const int32_t x = kept ? s.tok[j] : a.tokens[q0 + j];
                if (x < 0 || x >= a.vocab) continue;
                const int g = row.segment_of(x);
                if (g < g0 || g >= g1) continue;
                bool again = false;  // an earlier one was the same
                for (int i = cur + 1; i < j && !again; ++i) again = tried(i, cur, x);
                if (!again) atomicAdd(&s.segment[g - g0], 0ull - weight_of(kept ? capped(s.p[j]) : row.at(x)));
            }
            __syncthreads();
        }
        if (warp == 0) {
            u64 own = 0;
            for (int g = lane; g < g1 - g0; g += 32) own += s.segment[g];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(~0u, own, o);
            u64(*totals)[kMostCluster] = s.totals;
            if (ctas == 1) {
                if (lane == 0) totals[round & 1][0] = own;
            } else if (lane < ctas) {
                cg::cluster_group cluster = cg::this_cluster();
                *cluster.map_shared_rank(&totals[round & 1][rank], lane) = own;
            }
        }
        if (ctas == 1)
            __syncthreads();
        else
            cg::this_cluster().sync();
        if (tid == 0) {
            u64 all = 0, before = 0;
            for (int k = 0; k < ctas; ++k) {
                if (k < rank) before += s.totals[round & 1][k];
                all += s.totals[round & 1][k];
            }
            s.all = all, s.before = before;
        }
        ++round;
        __syncthreads();
    };

    // ---- the walk: tokens in order, 32 at a time, by the first warp of every CTA ----
    const bool drawn = a.draft_probs != nullptr;
    int cur = 0, count = 1, from = 1, base = 1;  // next token to look at, first of the window
    float c = 0.f;
    double over = 0., left = 1.;
    int32_t up = -1, tok = -1;
    float u = 0.f, pt = 0.f, qt = 0.f;
    bool stale = false;  // a token was turned down since `left` was summed
    auto window = [&]() {
        const int j = base + lane;
        up = -1, tok = -1, u = pt = qt = 0.f;
        if (j < n) {
            up = a.parents ? a.parents[q0 + j] : j - 1;
            tok = a.tokens[q0 + j];
            u = a.uniform[q0 + j];
            const bool ok = up >= 0 && up < j && tok >= 0 && tok < a.vocab;
            if (ok) {
                const int64_t row = q0 + up;
                pt = positive(to_f32(static_cast<const T *>(a.target_probs)[row * a.target_stride + tok]));
                if (drawn) qt = positive(to_f32(static_cast<const T *>(a.draft_probs)[row * a.draft_stride + tok]));
            } else {
                up = -1;
                if (rank == 0) report(a.err_word, SSD_DEVERR_METADATA);
            }
            if (kept) s.up[j] = up, s.tok[j] = tok, s.p[j] = pt;
        }
        __syncwarp();
    };
    if (warp == 0) {
        window();
        if (rank == 0) {
            for (int i = lane; i < a.max_path; i += 32) path[i] = i == 0 ? 0 : -1;
            __syncwarp();
        }
    }
    for (;;) {
        if (warp == 0) {
            bool wait = false, full = count >= a.max_path;
            while (!wait && !full) {
                const uint32_t next = __ballot_sync(~0u, up == cur && base + lane >= from);
                if (next == 0) {
                    base += 32;
                    if (base >= n) break;
                    window();
                    continue;
                }
                if (stale) {  // only a further token behind the same one needs the sum: in a chain there is none
                    wait = true;
                    break;
                }
                const int src = __ffs(next) - 1, j = base + src;
                const int32_t x = __shfl_sync(~0u, tok, src);
                const float uj = __shfl_sync(~0u, u, src), pj = __shfl_sync(~0u, pt, src), qj = __shfl_sync(~0u, qt, src);
                from = j + 1;
                bool takes;
                float rest = pj;
                if (drawn) {
                    rest = rest_of(pj, qj, c);
                    takes = __dmul_rn(__dmul_rn((double)uj, (double)qj), left) < (double)rest;
                } else {
                    // turned down before, behind the same token?  (the window's tokens are here)
                    bool again = up == cur && tok == x && lane < src;
                    if (cur + 1 < base)
                        for (int i = cur + 1 + lane; i < base; i += 32) again |= tried(i, cur, x);
                    if (__any_sync(~0u, again)) rest = 0.f;
                    takes = __dmul_rn((double)uj, left) < (double)rest;
                }
                if (takes) {
                    if (rank == 0 && lane == 0) path[count] = j;
                    ++count, cur = j;
                    c = 0.f, over = 0., left = 1.;
                    full = count >= a.max_path;
                } else if (drawn) {
                    over = __dadd_rn(over, left);
                    c = (float)over;
                    stale = true;
                } else {
                    left = fmax(__dsub_rn(left, (double)rest), 0.);
                }
            }
            if (lane == 0) s.cur = cur, s.count = count, s.c = c, s.more = wait, s.tried = !full;
        }
        __syncthreads();
        if (!s.more) break;
        {
            const Row<T> row(a, q0 + s.cur, s.c, true);
            sum_row(row, false, 0);
        }
        left = __dmul_rn(__ll2double_rn((long long)s.all), 1. / kUnit);
        stale = false;
        __syncthreads();
    }
    // ---- the next token ----
    cur = s.cur;
    c = s.c;
    bool drop = !drawn && s.tried;
    sum_row(Row<T>(a, q0 + cur, c, drawn && c > 0.f), drop, cur);
    if (s.all == 0 && (drop || c > 0.f)) {
        c = 0.f, drop = false;
        __syncthreads();
        sum_row(Row<T>(a, q0 + cur, 0.f, false), false, cur);
    }
    const Row<T> row(a, q0 + cur, c, drawn && c > 0.f);
    const u64 all = s.all, before = s.before;
    const u64 draw24 = (u64)min(max((long long)(draw * 16777216.f), 0ll), 16777215ll);
    const u64 mark = (all >> 24) * draw24 + (((all & 0xFFFFFFull) * draw24) >> 24);
    const int g0 = first_segment(row, rank), g1 = first_segment(row, rank + 1);
    const u64 own = s.totals[(round - 1) & 1][rank];
    if (rank == 0 && tid == 0) {
        a.path_lens[r] = s.count, a.accepted[r] = s.count - 1;
        if (all == 0) {
            a.next_tokens[r] = -1;
            report(a.err_word, SSD_DEVERR_METADATA);
        }
    }
    if (all > 0 && mark >= before && mark - before < own) {  // in this CTA's stretch
        if (warp == 0) {
            // the segment: 32 at a time
            u64 rest = mark - before;
            int found = -1;
            for (int g = g0; found < 0 && g < g1; g += 32) {
                const u64 w = g + lane < g1 ? s.segment[g + lane - g0] : 0;
                u64 sum = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 v = __shfl_up_sync(~0u, sum, o);
                    if (lane >= o) sum += v;
                }
                const uint32_t over_it = __ballot_sync(~0u, sum > rest);
                if (over_it) {
                    const int at = __ffs(over_it) - 1;
                    found = g + at;
                    rest -= __shfl_sync(~0u, sum - w, at);
                } else {
                    rest -= __shfl_sync(~0u, sum, 31);
                }
            }
            if (lane == 0) s.found = found, s.rest = rest;
            // its entries: those turned down are marked
            s.turned_down[lane] = 0;
            __syncwarp();
            if (drop)
                for (int j = cur + 1 + lane; j < n; j += 32) {
                    const int32_t x = kept ? s.tok[j] : a.tokens[q0 + j];
                    if (tried(j, cur, -1) && x >= 0 && x < a.vocab && row.segment_of(x) == found) {
                        const int at = x + row.shift - found * kSegment;
                        atomicOr(&s.turned_down[at >> 5], 1u << (at & 31));
                    }
                }
        }
        __syncthreads();
        // the entry: a warp has 32 N of the segment's
        constexpr int N = kVec<T>, kSteps = kSegment / (32 * N);
        static_assert(kSteps <= kWarps, "a step for each warp at most");
        const int found = s.found, at = (warp * 32 + lane) * N;  // in the segment
        u64 w[N], sum = 0, upto = 0;
        if (warp < kSteps) {
            float rests[N];
            row.get(found * kSegment - row.shift + at, rests);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                w[e] = s.turned_down[(at + e) >> 5] >> ((at + e) & 31) & 1 ? 0 : weight_of(rests[e]);
                sum += w[e];
            }
            upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) s.steps[warp] = upto;
        }
        __syncthreads();
        if (warp < kSteps) {
            u64 here = 0;
            for (int i = 0; i < warp; ++i) here += s.steps[i];
            if (s.rest >= here && s.rest - here < s.steps[warp]) {
                const u64 rest = s.rest - here;
                if (lane == __ffs(__ballot_sync(~0u, upto > rest)) - 1) {
                    u64 left_over = rest - (upto - sum);
                    int e = 0;
#pragma unroll
                    for (int k = 0; k < N - 1; ++k)
                        if (e == k && left_over >= w[k]) left_over -= w[k], ++e;
                    a.next_tokens[r] = found * kSegment - row.shift + at + e;
                }
            }
        }
    }
}

template <typename T> cudaError_t launch(const kv_verify_args &a, cudaStream_t s) {
    // CTAs of a request: as many as run at once, each with 2048 entries at least (256 chains of 65536 entries, again on the same rows, 19.8 us with 2,
    // 21.7 with one, 24.4 with 4: the walk costs each the same)
    int ctas = 1;
    while (ctas < kMostCluster && (int64_t)a.num_seqs * ctas * 2 <= 4ll * device_sms() && a.vocab / (ctas * 2) >= 2048) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.num_seqs * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kv_verify_kernel<T>, a, ctas);
}

}  // namespace

cudaError_t kv_verify_launch(const kv_verify_args &a, cudaStream_t s) {
    return a.dtype == SSD_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace ssd
