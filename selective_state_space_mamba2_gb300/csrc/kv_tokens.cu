// Per-token passes around the attention: kv_qk_norm_rope and kv_commit_tokens.
//
// Both are bound by HBM: every row is read once and written once in 16-byte pieces (two for
// fp32), 8 elements a lane.
#include "kv.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

// ---- kv_qk_norm_rope ---------------------------------------------------------
//
// n = x w / sqrt(mean(x^2) + eps) and the rotation of n are one linear map of x once the mean is
// known: y_e = r (a_e x_e + b_e x_p), with p the other entry of e's pair, a_e = w_e cos and
// b_e = -+ w_p sin (a_e = w_e, b_e = 0 beyond the rotated part).  a and b depend on the token and
// the weights alone, so a lane computes them once per token for its 8 entries and reuses them for
// every head; a row costs 8 squares, a shuffle reduction and 16 multiply-adds per lane.  CTAs walk
// over tokens, with the weights in shared memory and the next token's position fetched ahead.

// Where a pair's other entry is: among the lane's own 8 (interleaved), in another lane (pairs half a
// rotation apart, whole lanes of entries), or anywhere (read again from memory).
enum { kPairInside = 0, kPairLane = 1, kPairLoad = 2 };

constexpr int kQkShift = 7, kQkThreads = 1 << kQkShift;
// CTAs of an SM: what hides the loads' latency is warps (65536 tokens of 32 + 8 heads of 128, bf16: 312,
// 296, 295, 280 and 308 us with 4 to 8); fp32 and partners read again need more registers each.
constexpr int qk_ctas_per_sm(int pair, int elem) { return pair == kPairLoad || elem == 4 ? 5 : 7; }

// query rows that a lane group has in flight
constexpr int qk_rows(int pair, int elem) { return (pair == kPairLoad ? 2 : 4) / (elem == 4 ? 2 : 1); }

// 8 entries of a row as they lie in memory; get and set go by pairs, for packed fp32 arithmetic.
template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float2 get(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(int i, float2 v) {
        __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        w[i] = *reinterpret_cast<uint32_t *>(&b);
    }
};
template <> struct Row8<float> {
    uint32_t w[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const float *p) {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ float2 get(int i) const {
        return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    __device__ __forceinline__ void set(int i, float2 v) {
        w[2 * i] = __float_as_uint(v.x), w[2 * i + 1] = __float_as_uint(v.y);
    }
};

// A lane's 8 cosines and sines (the sine with its sign in y_e); 1 and 0 beyond the rotated part.
template <int PAIR>
__device__ __forceinline__ void angles(const kv_qk_args &a, int32_t pos, int e0, float (&cs)[8], float (&sn)[8]) {
    const int R = a.rotary_dim, half = R / 2;
    const float *row = a.cos_sin + (int64_t)pos * R;
    if (PAIR == kPairLoad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            cs[i] = 1.f, sn[i] = 0.f;
            if (e < R) {
                const bool low = a.interleaved ? (e & 1) == 0 : e < half;
                const int idx = a.interleaved ? e >> 1 : (low ? e : e - half);
                cs[i] = row[idx];
                sn[i] = low ? -row[half + idx] : row[half + idx];
            }
        }
    } else if (e0 < R) {  // 16-byte pieces; R is a multiple of 8 (inside) or 16 (lane)
        if (PAIR == kPairInside) {
            const float4 c = *reinterpret_cast<const float4 *>(row + e0 / 2);
            const float4 s = *reinterpret_cast<const float4 *>(row + half + e0 / 2);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[2 * i] = cs[2 * i + 1] = cc[i];
                sn[2 * i] = -ss[i], sn[2 * i + 1] = ss[i];
            }
        } else {
            const bool low = e0 < half;
            const float4 *c = reinterpret_cast<const float4 *>(row + (low ? e0 : e0 - half));
            const float4 *s = reinterpret_cast<const float4 *>(row + half + (low ? e0 : e0 - half));
            const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
            const float f = low ? -1.f : 1.f;
            cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
            sn[0] = f * s0.x, sn[1] = f * s0.y, sn[2] = f * s0.z, sn[3] = f * s0.w;
            sn[4] = f * s1.x, sn[5] = f * s1.y, sn[6] = f * s1.z, sn[7] = f * s1.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    }
}

// A row (head) is `width` lanes, 8 entries each (width: headdim / 8 rounded up to a power of two;
// WIDTH where the kernel is made for it, else 0).  A lane group loads its first key and value row and W
// query rows before it computes the first.
template <typename T, int PAIR, int WIDTH, bool kMany>
__global__ void __launch_bounds__(kQkThreads, qk_ctas_per_sm(PAIR, sizeof(T))) kv_qk_kernel(const kv_qk_args a, const int any_width, const int any_side) {
    constexpr int W = qk_rows(PAIR, sizeof(T));
    constexpr int kWords = 2 * (int)sizeof(T);  // 32-bit words of 8 entries
    __shared__ __align__(16) float weights[4][256];  // of q's entries and their partners, of k's
    const int width = WIDTH ? WIDTH : any_width;
    const int D = a.headdim, R = a.rotary_dim, half = R / 2;
    // kMany: 2^side_shift tokens side by side, whole warps each
    const int side_shift = kMany ? any_side : 0;
    const int per_shift = kQkShift - side_shift, in_token = threadIdx.x & ((1 << per_shift) - 1);
    const int sub = threadIdx.x & (width - 1), group = in_token / width, groups = (1 << per_shift) / width;
    const int e0 = sub * 8;
    const bool live = e0 < D;
    const bool want_k = a.k_out || a.k_cache;
    const bool turns = e0 < R;  // this lane's entries are (with kPairLoad: may be) rotated

    int src_lane = 0;  // kPairLane: whose entries are the partners of this lane's
    if (PAIR == kPairLane && turns) src_lane = (e0 < half ? e0 + half : e0 - half) / 8;
    auto partner = [&](int i) -> int {
        const int e = e0 + i;
        if (e >= R) return e;
        if (PAIR == kPairInside || (PAIR == kPairLoad && a.interleaved)) return e ^ 1;
        return e < half ? e + half : e - half;
    };
    if (threadIdx.x < width && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            weights[0][e0 + i] = a.q_weight ? a.q_weight[e0 + i] : 1.f;
            weights[1][e0 + i] = a.q_weight ? a.q_weight[partner(i)] : 1.f;
            weights[2][e0 + i] = a.k_weight ? a.k_weight[e0 + i] : 1.f;
            weights[3][e0 + i] = a.k_weight ? a.k_weight[partner(i)] : 1.f;
        }
    }
    __syncthreads();
    // a and b of this lane's entries for q (which = 0) or k (2)
    auto factors = [&](int which, const float (&cs)[8], const float (&sn)[8], float2 (&fa)[4], float2 (&fb)[4]) {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 w = *reinterpret_cast<const float4 *>(&weights[which][e0 + i]);
            const float4 o = *reinterpret_cast<const float4 *>(&weights[which + 1][e0 + i]);
            fa[i / 2] = tc::mul_f2(make_float2(cs[i], cs[i + 1]), make_float2(w.x, w.y));
            fa[i / 2 + 1] = tc::mul_f2(make_float2(cs[i + 2], cs[i + 3]), make_float2(w.z, w.w));
            fb[i / 2] = tc::mul_f2(make_float2(sn[i], sn[i + 1]), make_float2(o.x, o.y));
            fb[i / 2 + 1] = tc::mul_f2(make_float2(sn[i + 2], sn[i + 3]), make_float2(o.z, o.w));
        }
    };
    const float inv_d = 1.f / (float)D;

    auto fetch = [&](Row8<T> &x, float2 (&other)[4], const T *in, bool on) {
        x.clear();
        if (on && live) x.load(in + e0);
        if (PAIR == kPairLoad) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                other[i] = on && live ? make_float2(to_f32(in[partner(2 * i)]), to_f32(in[partner(2 * i + 1)]))
                                      : make_float2(0.f, 0.f);
        }
    };
    // one row: norm and rotation
    auto turn = [&](const Row8<T> &x, const float2 (&other)[4], const float2 (&fa)[4], const float2 (&fb)[4], bool norm) {
        float r = 1.f;
        if (norm) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = tc::fma_f2(x.get(i), x.get(i), s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (o < width) ss += __shfl_xor_sync(~0u, ss, o);
            r = rsqrtf(fmaf(ss, inv_d, a.eps));
        }
        Row8<T> p = x, y;
        if (PAIR == kPairLane) {
            // beyond the rotated part there is no partner: zero, whatever the other lane holds
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t v = __shfl_sync(~0u, x.w[i], src_lane, width);
                p.w[i] = turns ? v : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 o;
            if (PAIR == kPairInside) {
                o = make_float2(x.get(i).y, x.get(i).x);
                if (!turns) o = make_float2(0.f, 0.f);
            } else if (PAIR == kPairLane) {
                o = p.get(i);
            } else {
                o = other[i];
                if (e0 + 2 * i >= R) o.x = 0.f;
                if (e0 + 2 * i + 1 >= R) o.y = 0.f;
            }
            y.set(i, tc::mul_f2(make_float2(r, r), tc::fma_f2(fa[i], x.get(i), tc::mul_f2(fb[i], o))));
        }
        return y;
    };

    int t = (blockIdx.x << side_shift) + (threadIdx.x >> per_shift);
    const int stride = gridDim.x << side_shift;
    if (t >= a.total_tokens) return;
    int32_t pos = R > 0 ? a.positions[t] : 0;
    int32_t slot = a.k_cache ? a.slots[t] : -1;
    while (true) {
        const bool more = t < a.total_tokens - stride;
        const int t_next = more ? t + stride : t;
        const int32_t pos_next = R > 0 ? a.positions[t_next] : 0;
        const int32_t slot_next = a.k_cache ? a.slots[t_next] : -1;
        if (R > 0 && (pos < 0 || pos >= a.max_position)) {  // the same for whole warps
            if (in_token == 0) report(a.err_word, SSD_DEVERR_METADATA);
        } else {
            T *kc = nullptr, *vc = nullptr;
            if (slot >= 0) {
                const int32_t blk = slot / a.block_size;
                if (blk >= a.num_blocks) {
                    if (in_token == 0) report(a.err_word, SSD_DEVERR_SLOT);
                } else {
                    const int64_t at = (int64_t)blk * a.cache_block_stride +
                                       (int64_t)(slot - blk * a.block_size) * a.kv_heads * D;
                    kc = static_cast<T *>(a.k_cache) + at;
                    vc = static_cast<T *>(a.v_cache) + at;
                }
            }
            const T *qin = static_cast<const T *>(a.q) + (int64_t)t * a.q_stride;
            const T *kin = static_cast<const T *>(a.k) + (int64_t)t * a.k_stride;
            const T *vin = static_cast<const T *>(a.v) + (int64_t)t * a.v_stride;
            constexpr int kOther = PAIR == kPairLoad ? W : 1;
            Row8<T> xq[W], xk, xv;
            float2 oq[kOther][4], ok[4];
            fetch(xk, ok, kin + group * D, want_k && group < a.kv_heads);
            if (vc && live && group < a.kv_heads) xv.load(vin + group * D + e0);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int h = group + j * groups;
                fetch(xq[j], oq[PAIR == kPairLoad ? j : 0], qin + h * D, h < a.nheads);
            }
            float cs[8], sn[8];
            float2 fa[4] = {}, fb[4] = {};
            angles<PAIR>(a, pos, e0, cs, sn);
            if (PAIR == kPairLoad) __syncwarp();  // in place: partners are read before a row is overwritten

            if (want_k) {
                factors(2, cs, sn, fa, fb);
                T *out = static_cast<T *>(a.k_out) + (int64_t)t * a.kv_heads * D;
                for (int h0 = 0; h0 < a.kv_heads; h0 += groups) {
                    const int h = h0 + group;
                    const bool on = h < a.kv_heads;
                    if (h0 > 0) {
                        fetch(xk, ok, kin + h * D, on);
                        if (PAIR == kPairLoad) __syncwarp();
                    }
                    const Row8<T> o = turn(xk, ok, fa, fb, a.k_weight != nullptr);
                    if (on && live) {
                        if (a.k_out) o.store(out + h * D + e0);
                        if (kc) o.store(kc + h * D + e0);
                    }
                }
            }
            if (vc && live)
                for (int h = group; h < a.kv_heads; h += groups) {
                    if (h != group) xv.load(vin + h * D + e0);
                    xv.store(vc + h * D + e0);
                }
            factors(0, cs, sn, fa, fb);
            T *out = static_cast<T *>(a.q_out) + (int64_t)t * a.nheads * D;
            for (int h0 = 0; h0 < a.nheads; h0 += groups * W) {
                if (h0 > 0) {
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const int h = h0 + group + j * groups;
                        fetch(xq[j], oq[PAIR == kPairLoad ? j : 0], qin + h * D, h < a.nheads);
                    }
                    if (PAIR == kPairLoad) __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    // no row is left for any lane group (where all rows are full the test itself costs 1 %, or, with
                    // interleaved pairs, gains 14)
                    if ((kMany || PAIR == kPairInside) && j > 0 && h0 + j * groups >= a.nheads) break;
                    const int h = h0 + group + j * groups;
                    const Row8<T> o = turn(xq[j], oq[PAIR == kPairLoad ? j : 0], fa, fb, a.q_weight != nullptr);
                    if (h < a.nheads && live) o.store(out + h * D + e0);
                }
            }
        }
        if (!more) break;
        t = t_next, pos = pos_next, slot = slot_next;
    }
}

template <typename T, int PAIR> cudaError_t launch_qk(const kv_qk_args &a, cudaStream_t s) {
    int width = 1;
    while (width * 8 < a.headdim) width *= 2;
    const int most = qk_ctas_per_sm(PAIR, sizeof(T)) * device_sms();
    // Tokens of few heads go side by side, as many as have all their query rows in flight in the CTA, where there are
    // more tokens than CTAs: 8192 tokens of 8 heads of 64 29.1 to 11.2 us, 16384 of 32 62 to 45, 4096 of 16
    // heads of 128 18.6 to 13.7 (in the kernel for one token the shift would cost 65536 tokens of 32 281 to 314).
    int side_shift = 0;
    while (side_shift < 2 && a.total_tokens > most << side_shift &&
           a.nheads <= (kQkThreads / width >> (side_shift + 1)) * qk_rows(PAIR, sizeof(T)))
        ++side_shift;
    const int ctas = (a.total_tokens + (1 << side_shift) - 1) >> side_shift;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const auto kernel = width == 16  // headdim 72 to 128, the common ones: the reduction unrolled
                            ? (side_shift ? kv_qk_kernel<T, PAIR, 16, true> : kv_qk_kernel<T, PAIR, 16, false>)
                            : (side_shift ? kv_qk_kernel<T, PAIR, 0, true> : kv_qk_kernel<T, PAIR, 0, false>);
    kernel<<<grid, kQkThreads, 0, s>>>(a, width, side_shift);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_qk(const kv_qk_args &a, cudaStream_t s) {
    const bool pieces = (reinterpret_cast<uintptr_t>(a.cos_sin) & 15u) == 0;  // 16-byte loads of the angles
    if (a.interleaved && a.rotary_dim % 8 == 0 && pieces) return launch_qk<T, kPairInside>(a, s);
    if (!a.interleaved && a.rotary_dim % 16 == 0 && pieces) return launch_qk<T, kPairLane>(a, s);
    return launch_qk<T, kPairLoad>(a, s);
}

// ---- kv_commit_tokens ----------------------------------------------------------
//
// One CTA copies kRows rows of keys and of values; a thread loads all its pieces of them before it
// stores the first.

constexpr int kCommitThreads = 256;
constexpr int kRows = 4;

__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const kv_commit_args a, const int elem,
                                                                   const int64_t rows) {
    __shared__ int64_t src_row[kRows], dst_off[kRows];
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    const int row_bytes = a.kv_heads * a.headdim * elem, pieces = row_bytes / 16;

    if (a.context_out) {  // requests are dealt over the grid's threads
        for (int64_t r = (int64_t)blockIdx.x * kCommitThreads + tid; r < a.num_seqs;
             r += (int64_t)gridDim.x * kCommitThreads) {
            const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1];
            int32_t n = a.path ? a.path_lens[r] : q1 - q0;
            const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_tokens || n < 0 || n > q1 - q0 ||
                             (a.path && n > a.max_path);
            if (bad) report(a.err_word, SSD_DEVERR_METADATA);
            a.context_out[r] = a.context_lens[r] + (bad ? 0 : n);
        }
    }
    if (tid < kRows) {
        const int64_t row = row0 + tid;
        int64_t src = -1, dst = 0;
        if (row < rows) {
            int64_t token = row;  // whose slot the row goes to
            src = row;
            if (a.path) {
                const int64_t r = row / a.max_path;
                const int32_t i = (int32_t)(row - r * a.max_path);
                const int32_t q0 = a.cu_seqlens[r], q1 = a.cu_seqlens[r + 1], n = a.path_lens[r];
                src = -1;
                if (q0 < 0 || q1 < q0 || q1 > a.total_tokens || n < 0 || n > a.max_path || n > q1 - q0) {
                    report(a.err_word, SSD_DEVERR_METADATA);
                } else if (i < n) {
                    const int32_t j = a.path[row];
                    if (j < 0 || j >= q1 - q0) {
                        report(a.err_word, SSD_DEVERR_METADATA);
                    } else {
                        src = (int64_t)q0 + j;
                        token = (int64_t)q0 + i;
                    }
                }
            }
            if (src >= 0) {
                const int32_t slot = a.slots[token], blk = slot / a.block_size;
                if (slot < 0) {
                    src = -1;
                } else if (blk >= a.num_blocks) {
                    report(a.err_word, SSD_DEVERR_SLOT);
                    src = -1;
                } else {
                    dst = ((int64_t)blk * a.cache_block_stride +
                           (int64_t)(slot - blk * a.block_size) * a.kv_heads * a.headdim) * elem;
                }
            }
        }
        src_row[tid] = src;
        dst_off[tid] = dst;
    }
    __syncthreads();
    const char *kin = static_cast<const char *>(a.k_new), *vin = static_cast<const char *>(a.v_new);
    char *kout = static_cast<char *>(a.k_cache), *vout = static_cast<char *>(a.v_cache);
    for (int p = tid; p < 2 * pieces; p += kCommitThreads) {  // keys' pieces, then values'
        const bool val = p >= pieces;
        const char *in = val ? vin : kin;
        char *out = val ? vout : kout;
        const int64_t stride = (val ? a.v_stride : a.k_stride) * elem;
        const int at = (val ? p - pieces : p) * 16;
        uint4 x[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (src_row[j] >= 0) x[j] = *reinterpret_cast<const uint4 *>(in + src_row[j] * stride + at);
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (src_row[j] >= 0) *reinterpret_cast<uint4 *>(out + dst_off[j] + at) = x[j];
    }
}

}  // namespace

cudaError_t kv_qk_launch(const kv_qk_args &a, cudaStream_t s) {
    return a.dtype == SSD_BF16 ? launch_qk<__nv_bfloat16>(a, s) : launch_qk<float>(a, s);
}

cudaError_t kv_commit_launch(const kv_commit_args &a, cudaStream_t s) {
    const int64_t rows = a.path ? (int64_t)a.num_seqs * a.max_path : a.total_tokens;
    int64_t grid = (rows + kRows - 1) / kRows;
    if (grid < 1) grid = 1;  // context_out alone
    kv_commit_kernel<<<(unsigned)grid, kCommitThreads, 0, s>>>(a, a.dtype == SSD_BF16 ? 2 : 4, rows);
    return cudaGetLastError();
}

}  // namespace ssd
