// kv_commit_tokens_fp8 and kv_read_tokens_fp8: keys and values into a cache in 8 bits, and back.
#include "kv_fp8.cuh"

namespace ssd {
namespace {

using fp8::max_u16x2;

// 8 values of a row in registers
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // Largest magnitudes so far, two side by side: bits of bf16 compare as whole numbers, infinity and NaN are above any.
    using Top = uint32_t;
    __device__ __forceinline__ void fold(Top &top) const {
        top = max_u16x2(top, max_u16x2(max_u16x2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), max_u16x2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
    }
    __device__ __forceinline__ static float value(Top top) { return __uint_as_float(max(top << 16, top & 0xFFFF0000u)); }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    using Top = uint32_t;
    __device__ __forceinline__ void fold(Top &top) const {
        float v[8];
        get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    }
    __device__ __forceinline__ static float value(Top top) { return __uint_as_float(top); }
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ---- kv_commit_tokens_fp8 -----------------------------------------------------
//
// A block's scale has to cover all its rows, so one team of threads has all of a call's rows of a block, a head,
// and keys or values: it reads them once into registers, reduces their maximum, and writes codes.  Teams are of
// 32 to 256 threads by the most rows a block can get; a block with more than a team holds is read twice.
// Which (request, block) an item is follows from closed forms: with a path, every request is given the most
// blocks that max_path tokens can lie in; without, request r's items start at cu_seqlens[r] / b + 2 r.
// What an item is takes four dependent reads, so a CTA of a large call has several, found side by side, a lane an item
// (32768 tokens of 8 heads of 128 bf16 in blocks of 16: 67 us with one item a CTA, 37 to 39 now, 0.76 to 0.80 of the copy
// rate; it is bound by instructions beside it.  256 paths of up to 5 tokens 8 us, again on the same 6.2: latency).

constexpr int kThreads = 256;
// pieces of 8 values that a thread holds: with 8, whole blocks of 16 rows are a warp's, which costs less an item, but a
// path's addresses and 32-bit values then take too many registers for four CTAs on an SM
template <typename T, bool kPath> constexpr int HoldOf = sizeof(T) == 2 && !kPath ? 8 : 4;
constexpr int kCtas = 4;         // of an SM
constexpr int kMostItems = 16;   // of a CTA

struct Item {
    int32_t rows;  // new rows of the block (0: nothing to do)
    int32_t fill;  // rows that it holds already
    int32_t id;    // block
    int32_t q0, n; // the request's first packed row, its tokens
    int32_t i0;    // first of its tokens (steps of the path) that goes to the block
    int32_t r;
};

// kPath: with a path; kEven: a team's step is whole rows (pieces of a row divide its threads)
template <typename T, bool kPath, bool kEven>
__global__ void __launch_bounds__(kThreads, kCtas)
    kv_commit_fp8_kernel(const kv_commit_fp8_args a, const int team, const int path_blocks, const int items) {
    constexpr int kHold = HoldOf<T, kPath>;
    __shared__ float tops[2][kThreads / 32];
    __shared__ Item found[kMostItems];
    const int tid = threadIdx.x, lane = tid % team, D = a.headdim, pieces = D / 8, b = a.block_size;
    const bool val = blockIdx.z > 0;
    const int head = blockIdx.y * (kThreads / team) + tid / team;

    auto bad = [&](int32_t q0, int32_t q1, int32_t c, int32_t n) {
        return q0 < 0 || q1 < q0 || q1 > a.total_tokens || c < 0 || n < 0 || n > q1 - q0 || (a.path && n > a.max_path) ||
               (n > 0 && (int64_t)c + n > (int64_t)a.table_cols * b);
    };
    if (blockIdx.y == 0 && blockIdx.z == 0) {  // requests are dealt over the grid's threads
        for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < a.num_seqs; r += (int64_t)gridDim.x * kThreads) {
            const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1], c = a.context_lens[r];
            const int32_t n = a.path ? a.path_lens[r] : q1 - q0;
            const bool no = bad(q0, q1, c, n);
            if (a.context_out) a.context_out[r] = c + (no ? 0 : n);
            if (no) report(a.err_word, SSD_DEVERR_METADATA);
        }
    }
    if (tid < 32) {
        const long long at = (long long)blockIdx.x * items + tid;
        int r;
        long long k;
        if (a.path) {
            r = (int)min(at / path_blocks, (long long)a.num_seqs), k = at - (long long)r * path_blocks;
        } else {
            const auto first = [&](int i) { return (long long)(a.cu_seqlens[i] / b) + 2ll * i; };
            r = fp8::last_at_most(a.num_seqs, (long long)blockIdx.x * items, first);
            if (tid < items)
                while (r + 1 < a.num_seqs && first(r + 1) <= at) ++r;
            k = at - first(r);
            if (k < 0) r = a.num_seqs;  // before the first request's tokens
        }
        Item m = {};
        if (tid < items && r < a.num_seqs) {
            const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1], c = a.context_lens[r];
            const int32_t n = a.path ? a.path_lens[r] : q1 - q0;
            // (c + n is within the table row, whose positions fit 32 bits)
            if (!bad(q0, q1, c, n) && n > 0 && k <= (c + n - 1) / b - c / b) {
                const int32_t col = c / b + (int32_t)k, lo = max(c, col * b);
                m.id = a.block_table[(int64_t)r * a.table_cols + col];
                m.fill = lo - col * b, m.i0 = lo - c, m.q0 = q0, m.n = q1 - q0, m.r = r;
                m.rows = (int32_t)min((int64_t)c + n, ((int64_t)col + 1) * b) - lo;
                if (m.id < 0 || m.id >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    m.rows = 0;
                }
            }
        }
        if (tid < items) found[tid] = m;
    }
    __syncthreads();
    if (head >= a.kv_heads) return;  // a whole team, or all of its warps; teams wait for their own threads only
    const T *in = static_cast<const T *>(val ? a.v_new : a.k_new) + (int64_t)head * D;
    const int64_t stride = val ? a.v_stride : a.k_stride, row = (int64_t)a.kv_heads * D;
    const int tok0 = lane / pieces, piece0 = lane - tok0 * pieces, tok_step = team / pieces, piece_step = team - tok_step * pieces;
    const int64_t in_step = tok_step * stride, out_step = tok_step * row;
    Eight<T> x[kHold];
    int turn = 0;  // which of the two places for maxima: changes with every item worked on, not with those that are empty
    for (int item = 0; item < items; ++item) {
        const Item m = found[item];
        const int count = m.rows * pieces;
        if (count == 0) continue;
        const int32_t *path = kPath ? a.path + (int64_t)m.r * a.max_path + m.i0 : nullptr;
        uint8_t *page = static_cast<uint8_t *>(val ? a.v_cache : a.k_cache) + (int64_t)m.id * a.cache_block_stride + (int64_t)head * D;
        float *scale = (val ? a.v_scale : a.k_scale) + (int64_t)m.id * a.kv_heads + head;
        const float before = m.fill > 0 ? *scale : 0.f;
        const bool held = count <= kHold * team;
        // Goes over the pieces of this thread from piece `at` of the item on: f(j, token, piece), for those that exist.
        auto pieces_from = [&](int at, auto &&f) {
            int tok = tok0 + at / team * tok_step, piece = piece0;
            if (!kEven) {
                const int first = at + lane;
                tok = first / pieces, piece = first - tok * pieces;
            }
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                if (at + j * team + lane < count) f(j, tok, piece);
                tok += tok_step;
                if (!kEven) {
                    piece += piece_step;
                    if (piece >= pieces) piece -= pieces, ++tok;
                }
            }
        };
        uint32_t there = 0;  // kPath: which of the pieces are the request's
        auto load = [&](int at) {
            there = 0;
            const T *p = in + (int64_t)(m.q0 + m.i0 + tok0 + at / team * tok_step) * stride + piece0 * 8;
            pieces_from(at, [&](int j, int tok, int piece) {
                if (kPath) {
                    const int32_t k = path[tok];
                    if (k < 0 || k >= m.n) {
                        report(a.err_word, SSD_DEVERR_METADATA);
                        return;
                    }
                    there |= 1u << j;
                    x[j].load(in + (int64_t)(m.q0 + k) * stride + piece * 8);
                } else if (kEven) {
                    x[j].load(p + j * in_step);
                } else {
                    x[j].load(in + (int64_t)(m.q0 + m.i0 + tok) * stride + piece * 8);
                }
            });
        };
        auto is_there = [&](int j) { return !kPath || (there >> j & 1); };
        typename Eight<T>::Top bits = 0;
        for (int at = 0; at < count; at += kHold * team) {
            load(at);
            pieces_from(at, [&](int j, int, int) {
                if (is_there(j)) x[j].fold(bits);
            });
        }
        float top = Eight<T>::value(bits);
        const bool odd = !(top < INFINITY);  // something that is not finite: only the others count
        if (odd) {
            top = 0.f;
            for (int at = 0; at < count; at += kHold * team) {
                if (!held) load(at);
                pieces_from(at, [&](int j, int, int) {
                    float v[8];
                    x[j].get(v);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (is_there(j) && fabsf(v[e]) < INFINITY) top = fmaxf(top, fabsf(v[e]));
                });
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        if (team > 32) {  // (two places: a warp is a barrier ahead of another at most)
            if ((tid & 31) == 0) tops[turn][tid >> 5] = top;
            asm volatile("bar.sync %0, %1;" ::"r"(tid / team + 1), "r"(team) : "memory");
            for (int w = 0; w < team / 32; ++w) top = fmaxf(top, tops[turn][tid / team * (team / 32) + w]);
            turn ^= 1;
        }
        float now = fp8::scale_for(top);
        if (m.fill > 0) {
            if (before >= now) {
                now = before;
            } else {  // the rows that are there already, by the larger scale
                const float ratio = before / now;
                for (int at = lane; at < m.fill * pieces; at += team) {
                    const int t = at / pieces;
                    uint2 *p = reinterpret_cast<uint2 *>(page + t * row) + (at - t * pieces);
                    float v[8];
                    fp8::decode8(*p, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= ratio;
                    *p = fp8::encode8(v);
                }
            }
        }
        __syncwarp();  // all have read the old one (wider teams have met above)
        if (lane == 0) *scale = now;
        const float inv = __frcp_rn(now);
        for (int at = 0; at < count; at += kHold * team) {
            if (!held) load(at);
            uint8_t *to = page + (m.fill + tok0 + at / team * tok_step) * row + piece0 * 8;
            pieces_from(at, [&](int j, int tok, int piece) {
                if (!is_there(j)) return;
                float v[8];
                x[j].get(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= inv;
                *reinterpret_cast<uint2 *>(kEven ? to + j * out_step : page + (m.fill + tok) * row + piece * 8) = fp8::encode8(v);
            });
            if (odd)  // once more: an infinity becomes NaN, not the largest value
                pieces_from(at, [&](int j, int tok, int piece) {
                    if (!is_there(j)) return;
                    float v[8];
                    x[j].get(v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], 0.f, v[e] * inv);
                    *reinterpret_cast<uint2 *>(page + (m.fill + tok) * row + piece * 8) = fp8::encode8(v);
                });
        }
    }
}

// ---- kv_read_tokens_fp8 -----------------------------------------------------------
//
// A CTA has the rows of kReadTokens packed tokens, keys and values; a thread has kFlight pieces of kCodes codes on their
// way at a time (16, or 8 where a head's size is no multiple of 16).  Bound by HBM: 16 prefixes of 500 to 8192 tokens of 8
// heads of 128 to bf16, 346 MB, 62 us, 0.82 of the copy rate (8 codes a piece: 73 us).

constexpr int kReadTokens = 8;
constexpr int kFlight = 4;

template <typename T, int kCodes> __global__ void __launch_bounds__(kThreads) kv_read_fp8_kernel(const kv_read_fp8_args a) {
    __shared__ int32_t ids[kReadTokens];      // block, -1: zeros, -2: nothing to write
    __shared__ int32_t offs[kReadTokens];     // row in the block
    const int tid = threadIdx.x, b = a.block_size;
    auto bad = [&](int32_t q0, int32_t q1, int32_t c) {
        return q0 < 0 || q1 < q0 || q1 > a.total_tokens || c < 0 ||
               (q1 > q0 && (int64_t)c + (q1 - q0) > (int64_t)a.table_cols * b);
    };
    for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < a.num_seqs; r += (int64_t)gridDim.x * kThreads)
        if (bad(a.cu_seqlens[r], a.cu_seqlens[r + 1], a.starts ? a.starts[r] : 0)) report(a.err_word, SSD_DEVERR_METADATA);
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    if (tid < 32) {
        int r = fp8::last_at_most(a.num_seqs, t0, [&](int i) { return (long long)a.cu_seqlens[i]; });
        if (tid < kReadTokens) {
            const int64_t t = t0 + tid;
            int32_t id = -2, off = 0;
            // the last request that starts at or before t (empty ones start where the next does)
            while (r + 1 < a.num_seqs && a.cu_seqlens[r + 1] <= t) ++r;
            const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1], c = a.starts ? a.starts[r] : 0;
            if (!bad(q0, q1, c) && t >= q0 && t < q1) {
                const int32_t pos = c + (int32_t)(t - q0), col = pos / b;
                off = pos - col * b;
                id = a.block_table[(int64_t)r * a.table_cols + col];
                if (id < 0 || id >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    id = -1;
                }
            }
            ids[tid] = id;
            offs[tid] = off;
        }
    }
    __syncthreads();
    constexpr int kWords = kCodes / 4;
    const int row = a.kv_heads * a.headdim, pieces = row / kCodes, per_head = a.headdim / kCodes;
    const int all = 2 * kReadTokens * pieces;  // keys of the tokens, then values
    for (int p0 = tid; p0 < all; p0 += kThreads * kFlight) {
        uint32_t c[kFlight][kWords];
        float s[kFlight];
        int64_t to[kFlight];
        bool val[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int p = p0 + j * kThreads;
            to[j] = -1;
            if (p >= all) continue;
            const int line = p / pieces, piece = p - line * pieces;
            val[j] = line >= kReadTokens;
            const int t = line - (val[j] ? kReadTokens : 0), id = ids[t];
            if (id == -2) continue;
            to[j] = (t0 + t) * row + piece * kCodes;
#pragma unroll
            for (int e = 0; e < kWords; ++e) c[j][e] = 0;
            s[j] = 0.f;
            if (id >= 0) {
                const uint8_t *from = static_cast<const uint8_t *>(val[j] ? a.v_cache : a.k_cache) +
                                      (int64_t)id * a.cache_block_stride + (int64_t)offs[t] * row + piece * kCodes;
                if constexpr (kCodes == 16) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(from));
                    c[j][0] = u.x, c[j][1] = u.y, c[j][2] = u.z, c[j][3] = u.w;
                } else {
                    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(from));
                    c[j][0] = u.x, c[j][1] = u.y;
                }
                s[j] = __ldg((val[j] ? a.v_scale : a.k_scale) + (int64_t)id * a.kv_heads + piece / per_head);
            }
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            if (to[j] < 0) continue;
            T *out = static_cast<T *>(val[j] ? a.v_out : a.k_out) + to[j];
#pragma unroll
            for (int h = 0; h < kCodes / 8; ++h) {
                float v[8];
                fp8::decode8(make_uint2(c[j][2 * h], c[j][2 * h + 1]), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= s[j];
                store8(out + 8 * h, v);
            }
        }
    }
}

int64_t ceil_div64(int64_t n, int64_t d) { return (n + d - 1) / d; }

}  // namespace

cudaError_t kv_commit_fp8_launch(const kv_commit_fp8_args &a, cudaStream_t s) {
    // most rows that a call brings to a block
    const int64_t most = a.path ? a.max_path : a.total_tokens, rows = most < a.block_size ? most : a.block_size;
    const bool bf16 = a.dtype == SSD_BF16;
    const int hold = a.path ? HoldOf<float, true> : bf16 ? HoldOf<__nv_bfloat16, false> : HoldOf<float, false>;
    int team = 32;
    while (team < kThreads && (rows * (a.headdim / 8) > (int64_t)team * hold || kThreads / team >= 2 * a.kv_heads)) team *= 2;
    int64_t items, path_blocks = 1;
    if (a.path) {
        path_blocks = (most + 2 * (int64_t)a.block_size - 2) / a.block_size;  // n tokens from any row of a block on
        items = path_blocks * a.num_seqs;
    } else {
        items = a.total_tokens / a.block_size + 2 * (int64_t)a.num_seqs;
    }
    if (items < 1) items = 1;  // context_out alone
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    // As many items to a CTA as let all CTAs run at once; they are blocks side by side.
    const int64_t side = ceil_div64(a.kv_heads, kThreads / team) * 2, share = ceil_div64(items * side, (int64_t)kCtas * device_sms());
    const int each = (int)(share < kMostItems ? share : kMostItems);
    const dim3 grid((unsigned)ceil_div64(items, each), (unsigned)(side / 2), 2);
    const bool even = team % (a.headdim / 8) == 0;
    const auto kernel = a.path ? (bf16 ? kv_commit_fp8_kernel<__nv_bfloat16, true, false> : kv_commit_fp8_kernel<float, true, false>)
                        : even ? (bf16 ? kv_commit_fp8_kernel<__nv_bfloat16, false, true> : kv_commit_fp8_kernel<float, false, true>)
                               : (bf16 ? kv_commit_fp8_kernel<__nv_bfloat16, false, false> : kv_commit_fp8_kernel<float, false, false>);
    kernel<<<grid, kThreads, 0, s>>>(a, team, (int)path_blocks, each);
    return cudaGetLastError();
}

cudaError_t kv_read_fp8_launch(const kv_read_fp8_args &a, cudaStream_t s) {
    const unsigned grid = (unsigned)ceil_div64(a.total_tokens, kReadTokens);
    const bool wide = a.headdim % 16 == 0 && a.cache_block_stride % 16 == 0;
    const auto kernel = a.dtype == SSD_BF16 ? (wide ? kv_read_fp8_kernel<__nv_bfloat16, 16> : kv_read_fp8_kernel<__nv_bfloat16, 8>)
                                            : (wide ? kv_read_fp8_kernel<float, 16> : kv_read_fp8_kernel<float, 8>);
    kernel<<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ssd
