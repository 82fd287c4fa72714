// Per-token passes around the attention: kv_qk_norm_rope and kv_commit_tokens.
//
// Both are bound by HBM: every row is read once and written once in 16-byte pieces (two for
// fp32), 8 elements a lane.
#include "kv.cuh"

namespace ssd {
namespace {

// ---- kv_qk_norm_rope ---------------------------------------------------------
//
// n = x w / sqrt(mean(x^2) + eps) and the rotation of n are one linear map of x once the mean is
// known: y_e = r (a_e x_e + b_e x_p), with p the other entry of e's pair, a_e = w_e cos and
// b_e = -+ w_p sin (a_e = w_e, b_e = 0 beyond the rotated part).  a and b depend on the token and
// the weights alone, so a lane computes them once for its 8 entries and reuses them for every
// head; a row costs 8 squares, a shuffle reduction and 16 multiply-adds per lane.

enum { kPairInside = 0, kPairLane = 1, kPairLoad = 2 };  // where a pair's other entry is

constexpr int kQkThreads = 128;

template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = u; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&v);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ Row8 from_lane(int src, int width) const {
        Row8 o;
        o.u.x = __shfl_sync(~0u, u.x, src, width);
        o.u.y = __shfl_sync(~0u, u.y, src, width);
        o.u.z = __shfl_sync(~0u, u.z, src, width);
        o.u.w = __shfl_sync(~0u, u.w, src, width);
        return o;
    }
};
template <> struct Row8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ Row8 from_lane(int src, int width) const {
        float f[8];
        get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __shfl_sync(~0u, f[i], src, width);
        Row8 o;
        o.set(f);
        return o;
    }
};

// One CTA per token; a row (head) is `width` lanes, 8 entries each (width: headdim / 8 rounded up
// to a power of two).  W heads of a lane group are loaded before the first is computed.
template <typename T, int PAIR>
__global__ void __launch_bounds__(kQkThreads) kv_qk_kernel(const kv_qk_args a, const int width) {
    constexpr int W = 4;
    const int t = blockIdx.x;
    const int D = a.headdim, R = a.rotary_dim, half = R / 2;
    const int sub = threadIdx.x & (width - 1), group = threadIdx.x / width, groups = kQkThreads / width;
    const int e0 = sub * 8;
    const bool live = e0 < D;

    int32_t pos = 0;
    if (R > 0) {
        pos = a.positions[t];
        if (pos < 0 || pos >= a.max_position) {  // the same for the whole CTA
            if (threadIdx.x == 0) report(a.err_word, SSD_DEVERR_METADATA);
            return;
        }
    }
    T *kc = nullptr, *vc = nullptr;
    if (a.k_cache) {
        const int32_t slot = a.slots[t];
        if (slot >= 0) {
            const int32_t blk = slot / a.block_size;
            if (blk >= a.num_blocks) {
                if (threadIdx.x == 0) report(a.err_word, SSD_DEVERR_SLOT);
            } else {
                const int64_t at = (int64_t)blk * a.cache_block_stride +
                                   (int64_t)(slot - blk * a.block_size) * a.kv_heads * D;
                kc = static_cast<T *>(a.k_cache) + at;
                vc = static_cast<T *>(a.v_cache) + at;
            }
        }
    }

    // this lane's cosines and sines, and which entry is each one's partner
    float cs[8], sn[8];
    int partner[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        cs[i] = 1.f, sn[i] = 0.f, partner[i] = e;
        if (e < R) {
            const bool low = PAIR == kPairInside ? (e & 1) == 0 : e < half;
            const int idx = PAIR == kPairInside ? e >> 1 : (low ? e : e - half);
            const float *row = a.cos_sin + (int64_t)pos * R;
            cs[i] = row[idx];
            sn[i] = low ? -row[half + idx] : row[half + idx];
            partner[i] = PAIR == kPairInside ? e ^ 1 : (low ? e + half : e - half);
        }
    }
    const int src_lane = PAIR == kPairLane ? min(partner[0] / 8, width - 1) : 0;

    for (int part = 0; part < 2; ++part) {
        const bool is_q = part == 0;
        const int heads = is_q ? a.nheads : a.kv_heads;
        T *out = static_cast<T *>(is_q ? a.q_out : a.k_out);
        if (!is_q && !out && !kc) break;
        const float *w = is_q ? a.q_weight : a.k_weight;
        float fa[8], fb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            fa[i] = cs[i], fb[i] = sn[i];
            if (w && live) {
                fa[i] *= w[e0 + i];
                fb[i] *= w[partner[i]];
            }
        }
        const T *in = static_cast<const T *>(is_q ? a.q : a.k) + (int64_t)t * (is_q ? a.q_stride : a.k_stride);
        for (int h0 = 0; h0 < heads; h0 += groups * W) {
            Row8<T> x[W];
            float other[PAIR == kPairLoad ? W : 1][8];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int h = h0 + j * groups + group;
                if (h < heads && live) {
                    x[j].load(in + h * D + e0);
                    if (PAIR == kPairLoad) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) other[j][i] = to_f32(in[h * D + partner[i]]);
                    }
                } else {
                    float z[8] = {};
                    x[j].set(z);
                    if (PAIR == kPairLoad) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) other[j][i] = 0.f;
                    }
                }
            }
            if (PAIR == kPairLoad) __syncwarp();  // in place: partners are read before a row is overwritten
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int h = h0 + j * groups + group;
                float v[8], y[8];
                x[j].get(v);
                float r = 1.f;
                if (w) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
                    for (int o = width / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                    r = rsqrtf(ss / (float)D + a.eps);
                }
                float p[8];
                if (PAIR == kPairInside) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = v[i ^ 1];
                } else if (PAIR == kPairLane) {
                    x[j].from_lane(src_lane, width).get(p);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = other[j][i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // beyond the rotated part the partner is the entry itself, and is left out
                    const float turned = e0 + i < R ? fb[i] * p[i] : 0.f;
                    y[i] = r * fmaf(fa[i], v[i], turned);
                }
                if (h < heads && live) {
                    Row8<T> o;
                    o.set(y);
                    if (out) o.store(out + ((int64_t)t * heads + h) * D + e0);
                    if (!is_q && kc) o.store(kc + h * D + e0);
                }
            }
        }
    }
    if (vc && live) {
        const T *in = static_cast<const T *>(a.v) + (int64_t)t * a.v_stride;
        for (int h = group; h < a.kv_heads; h += groups) {
            Row8<T> x;
            x.load(in + h * D + e0);
            x.store(vc + h * D + e0);
        }
    }
}

template <typename T> cudaError_t launch_qk(const kv_qk_args &a, cudaStream_t s) {
    int width = 1;
    while (width * 8 < a.headdim) width *= 2;
    const dim3 grid((unsigned)a.total_tokens);
    if (a.interleaved)
        kv_qk_kernel<T, kPairInside><<<grid, kQkThreads, 0, s>>>(a, width);
    else if (a.rotary_dim % 16 == 0)
        kv_qk_kernel<T, kPairLane><<<grid, kQkThreads, 0, s>>>(a, width);
    else
        kv_qk_kernel<T, kPairLoad><<<grid, kQkThreads, 0, s>>>(a, width);
    return cudaGetLastError();
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
