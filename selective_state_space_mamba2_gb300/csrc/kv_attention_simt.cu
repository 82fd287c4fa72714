// kv_tree_attention on the CUDA cores, in fp32: every type, head size, group and page size the
// tensor-core kernel does not take, and the kernel that joins the parts of cut items.
//
// Online softmax over key tiles of 32 for 16 query rows a CTA: keys and values of a tile are
// staged in shared memory as fp32, a thread owns one row's 4 scores of a tile and an eighth of
// its output.  Bound by shared-memory reads (one 16-byte read for 4 multiply-adds); its use is
// fp32 decode, where few rows meet each key.
#include "kv_sched.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kRowTile = 16;
constexpr int kKeyShift = 5;
constexpr int kKeyTile = 1 << kKeyShift;
constexpr int kOverhead = 1;  // of an item, in key tiles
constexpr int kMinUnits = 4;
constexpr int kCtasPerSm = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int smem_bytes(int D) { return (kRowTile * (D + 4) + 2 * kKeyTile * (D + 4) + kRowTile * (kKeyTile + 1)) * 4; }

template <typename T> __device__ __forceinline__ void load8(float (&f)[8], const T *p);
template <> __device__ __forceinline__ void load8<float>(float (&f)[8], const float *p) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(float (&f)[8], const __nv_bfloat16 *p) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// NV: 32-float pieces of a row a thread group covers, headdim <= 32 NV
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) kv_attention_simt_kernel(const kv_attention_args a, const kvs::Parts parts,
                                                                  const kvs::Tiling g) {
    extern __shared__ __align__(16) float smem[];
    __shared__ kvs::FindSmem find;
    const int D = a.headdim, group = a.nheads / a.kv_heads, pitch = D + 4;
    float *sq = smem, *sk = sq + kRowTile * pitch, *sv = sk + kKeyTile * pitch, *sp = sv + kKeyTile * pitch;
    const int tid = threadIdx.x, row = tid >> 3, sub = tid & 7;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join kernel may be set up
    kvs::Walk w;
    if (!kvs::find_run(a, g, kMinUnits, find, parts.borders, w)) return;
    const float c = a.scale * kLog2e;
    const int pieces = D / 8;
    bool more = true;
    while (more) {
        const int heads = w.heads(g, group), rows = w.tokens(g) * heads, head0 = w.h * group + w.part * g.heads;
        const int token0 = w.first_token(g);
        // query rows
        __syncthreads();
        for (int i = tid; i < kRowTile * pieces; i += kThreads) {
            const int r = i / pieces, e = (i % pieces) * 8;
            float f[8] = {};
            if (r < rows) {
                const int64_t tok = w.q.q0 + token0 + r / heads;
                load8(f, static_cast<const T *>(a.q) + tok * a.q_stride + (head0 + r % heads) * D + e);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq[r * pitch + e + j] = f[j];
        }
        const int32_t my_tok = row < rows ? token0 + row / heads : -1;
        const uint32_t *mask = a.tree_mask && my_tok >= 0 ? a.tree_mask + (int64_t)(w.q.q0 + my_tok) * a.mask_words : nullptr;

        float top = -INFINITY, sum = 0.f, acc[NV][4] = {};
        for (int t = w.t0; t < w.t1; ++t) {
            const bool cached = t < w.cached_tiles;
            const int32_t base = (cached ? t : t - w.cached_tiles) * kKeyTile;
            const int32_t limit = cached ? w.q.c : w.new_seen;  // keys from here on do not exist
            __syncthreads();
            for (int i = tid; i < kKeyTile * pieces; i += kThreads) {
                const int key = i / pieces, e = (i % pieces) * 8;
                const int32_t pos = base + key;
                float fk[8] = {}, fv[8] = {};
                if (pos < limit) {
                    if (cached) {
                        const int32_t col = pos / a.block_size;
                        const int32_t id = a.block_table[(int64_t)w.r * a.table_cols + col];
                        if (id >= 0 && id < a.num_blocks) {
                            const int64_t at = (int64_t)id * a.cache_block_stride +
                                               ((int64_t)(pos - col * a.block_size) * a.kv_heads + w.h) * D + e;
                            load8(fk, static_cast<const T *>(a.k_cache) + at);
                            load8(fv, static_cast<const T *>(a.v_cache) + at);
                        } else if (e == 0) {
                            report(a.err_word, SSD_DEVERR_SLOT);
                        }
                    } else {
                        const int64_t tok = w.q.q0 + pos;
                        load8(fk, static_cast<const T *>(a.k_new) + tok * a.k_stride + w.h * D + e);
                        load8(fv, static_cast<const T *>(a.v_new) + tok * a.v_stride + w.h * D + e);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sk[key * pitch + e + j] = fk[j];
                    sv[key * pitch + e + j] = fv[j];
                }
            }
            __syncthreads();
            // scores of keys sub + 8 j
            float s[4] = {};
            for (int e = 0; e < D; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(sq + row * pitch + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 y = *reinterpret_cast<const float4 *>(sk + (sub + 8 * j) * pitch + e);
                    s[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[j]))));
                }
            }
            float best = -INFINITY;
            bool sees[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t pos = base + sub + 8 * j;
                sees[j] = pos < limit && my_tok >= 0;
                if (!cached && sees[j])
                    sees[j] = mask ? (mask[pos >> 5] >> (pos & 31)) & 1u : pos <= my_tok;
                s[j] = sees[j] ? s[j] * c : -INFINITY;
                best = s[j] > best || s[j] != s[j] ? s[j] : best;
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                const float v = __shfl_xor_sync(~0u, best, o);
                best = v > best || v != v ? v : best;
            }
            const float now = best > top || best != best ? best : top;
            const float from = now == -INFINITY ? 0.f : now;  // nothing seen yet: weights are exp2(-inf) = 0
            const float shrink = exp2f(top - from);
            top = now;
            sum *= shrink;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[j] - from);
                sp[row * (kKeyTile + 1) + sub + 8 * j] = sees[j] ? p : 0.f;
                sum += sees[j] ? p : 0.f;
            }
            __syncwarp();  // a row's weights are written and read by the same warp
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[v][j] *= shrink;
            for (int key = 0; key < kKeyTile; ++key) {
                const float p = sp[row * (kKeyTile + 1) + key];
                if (p == 0.f) continue;  // not seen: its value stays out, whatever it is
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int e = 32 * v + 4 * sub;
                    if (e < D) {
                        const float4 y = *reinterpret_cast<const float4 *>(sv + key * pitch + e);
                        acc[v][0] = fmaf(p, y.x, acc[v][0]);
                        acc[v][1] = fmaf(p, y.y, acc[v][1]);
                        acc[v][2] = fmaf(p, y.z, acc[v][2]);
                        acc[v][3] = fmaf(p, y.w, acc[v][3]);
                    }
                }
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (my_tok >= 0) {
            if (w.whole()) {
                const int64_t out_row = (int64_t)(w.q.q0 + my_tok) * a.nheads + head0 + row % heads;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw nothing: zeros
                T *out = static_cast<T *>(a.out) + out_row * D;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int e = 32 * v + 4 * sub;
                    if (e < D)
#pragma unroll
                        for (int j = 0; j < 4; ++j) out[e + j] = from_f32<T>(acc[v][j] * inv);
                }
                if (a.lse && sub == 0) a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                const int64_t part = ((int64_t)blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1)) * g.rows + row;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int e = 32 * v + 4 * sub;
                    if (e < D) *reinterpret_cast<float4 *>(parts.sums + part * D + e) =
                        make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
                }
                if (sub == 0) parts.stats[part] = make_float2(top, sum);
            }
        }
        more = w.next(a, g);
    }
}

// ---- joining the parts of a cut item -----------------------------------------------
//
// One row of CTAs per border: where the border before CTA b's run is the first to cut an item, its
// parts are added up, that of CTA b - 1 (which began the item) and those of the CTAs from b on:
//   out = sum_i 2^(m_i - m) O_i / L,  L = sum_i 2^(m_i - m) l_i,  m = max_i m_i.
// Bound by the latency of three dependent reads (border, statistics, sums).  kSplit warps share a
// row's parts: 4 for decode's few rows, whose items may have dozens of parts (65536 keys of one
// request: 38), 1 for prompts' many rows of two or three parts.
constexpr int kJoinThreads = 128;
constexpr int kSplitRows = 16;  // tiles of at most so many rows are joined by 4 warps a row

template <typename T, int NV, int kSplit>  // NV: 128-float pieces of a row
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const kv_attention_args a, const kvs::Parts parts,
                                                               const kvs::Tiling g) {
    __shared__ float part_acc[kSplit][NV * 128];
    __shared__ float part_sum[kSplit];
    const int D = a.headdim, b = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = kSplit > 1 ? blockIdx.y : blockIdx.y * 4 + warp, share = kSplit > 1 ? warp : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are complete
    const kvs::Border me = parts.borders[b];
    const int n = me.parts;
    if (n == 0 || row >= me.tokens * me.heads) return;
    // part k: of CTA b - 1 + k
    auto part_row = [&](int k) { return ((int64_t)(b - 1 + k) * 2 + (k == 0 ? 1 : 0)) * g.rows + row; };
    float top = -INFINITY;
    for (int k = lane; k < n; k += 32) {
        const float m = parts.stats[part_row(k)].x;
        top = m > top || m != m ? m : top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(~0u, top, o);
        top = m > top || m != m ? m : top;
    }
    const float from = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[NV][4] = {};
    // parts share, share + kSplit, ...: 32 a round, a lane each for the factors
    for (int k0 = share; k0 < n; k0 += 32 * kSplit) {
        const int mine = k0 + lane * kSplit;
        float f = 0.f;
        if (mine < n) {
            const float2 st = parts.stats[part_row(mine)];
            f = exp2f(st.x - from);
            sum = fmaf(f, st.y, sum);
        }
        const int here = min(32, (n - k0 + kSplit - 1) / kSplit);
        for (int i0 = 0; i0 < here; i0 += 4) {  // four loads in flight, the last ones repeated with factor 0
            float4 v[4][NV];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *src = parts.sums + part_row(k0 + min(i0 + i, here - 1) * kSplit) * D;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    v[i][j] = 128 * j + 4 * lane < D ? *reinterpret_cast<const float4 *>(src + 128 * j + 4 * lane)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float fk = __shfl_sync(~0u, f, i0 + i < here ? i0 + i : 0);
                if (i0 + i < here) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        acc[j][0] = fmaf(fk, v[i][j].x, acc[j][0]);
                        acc[j][1] = fmaf(fk, v[i][j].y, acc[j][1]);
                        acc[j][2] = fmaf(fk, v[i][j].z, acc[j][2]);
                        acc[j][3] = fmaf(fk, v[i][j].w, acc[j][3]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (kSplit > 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            *reinterpret_cast<float4 *>(&part_acc[share][128 * j + 4 * lane]) =
                make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        if (lane == 0) part_sum[share] = sum;
        __syncthreads();
        if (warp > 0) return;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kSplit; ++w) sum += part_sum[w];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kSplit; ++w) {
                const float4 v = *reinterpret_cast<const float4 *>(&part_acc[w][128 * j + 4 * lane]);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            acc[j][0] = s.x, acc[j][1] = s.y, acc[j][2] = s.z, acc[j][3] = s.w;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out_row = (int64_t)(me.token0 + row / me.heads) * a.nheads + me.head0 + row % me.heads;
    T *out = static_cast<T *>(a.out) + out_row * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = 128 * j + 4 * lane;
        if (e < D) {
            if (sizeof(T) == 4) {
                *reinterpret_cast<float4 *>(out + e) =
                    make_float4(acc[j][0] * inv, acc[j][1] * inv, acc[j][2] * inv, acc[j][3] * inv);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) out[e + i] = from_f32<T>(acc[j][i] * inv);
            }
        }
    }
    if (a.lse && lane == 0) a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <typename T, int NV>
cudaError_t launch_join(const kv_attention_args &a, const kvs::Parts &p, int grid, const kvs::Tiling &g, cudaStream_t s) {
    // a programmatic dependent of the attention kernel: its CTAs may be set up while that ends
    const bool split = g.rows <= kSplitRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)(split ? g.rows : kvs::ceil_div(g.rows, 4)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return split ? cudaLaunchKernelEx(&cfg, kv_join_kernel<T, NV, 4>, a, p, g)
                 : cudaLaunchKernelEx(&cfg, kv_join_kernel<T, NV, 1>, a, p, g);
}

kvs::Tiling simt_tiling(const kv_attention_args &a) { return kvs::tiling(a, kRowTile, kKeyShift, kOverhead); }

int simt_grid(const kv_attention_args &a, const kvs::Tiling &g) {
    return kvs::grid_of(a, g, kMinUnits, kCtasPerSm * device_sms());
}

template <typename T, int NV>
cudaError_t launch(const kv_attention_args &a, void *ws, cudaStream_t s) {
    const kvs::Tiling g = simt_tiling(a);
    const int grid = simt_grid(a, g);
    const kvs::Parts parts = kvs::parts_at(ws, grid, g.rows, a.headdim);
    const int smem = smem_bytes(a.headdim);
    cudaError_t e = cudaFuncSetAttribute(kv_attention_simt_kernel<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kv_attention_simt_kernel<T, NV><<<grid, kThreads, smem, s>>>(a, parts, g);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kvs::join_launch(a, parts, grid, g, s);
}

template <typename T> cudaError_t launch_dim(const kv_attention_args &a, void *ws, cudaStream_t s) {
    if (a.headdim <= 64) return launch<T, 2>(a, ws, s);
    if (a.headdim <= 128) return launch<T, 4>(a, ws, s);
    return launch<T, 8>(a, ws, s);
}

}  // namespace

cudaError_t kvs::join_launch(const kv_attention_args &a, const Parts &p, int grid, const Tiling &g, cudaStream_t s) {
    if (grid < 2) return cudaSuccess;
    if (a.dtype == SSD_BF16)
        return a.headdim <= 128 ? launch_join<__nv_bfloat16, 1>(a, p, grid, g, s)
                                : launch_join<__nv_bfloat16, 2>(a, p, grid, g, s);
    return a.headdim <= 128 ? launch_join<float, 1>(a, p, grid, g, s) : launch_join<float, 2>(a, p, grid, g, s);
}

size_t kv_attention_simt_workspace(const kv_attention_args &a) {
    const kvs::Tiling g = simt_tiling(a);
    return kvs::parts_bytes(simt_grid(a, g), g.rows, a.headdim);
}

cudaError_t kv_attention_simt_launch(const kv_attention_args &a, void *ws, cudaStream_t s) {
    return a.dtype == SSD_BF16 ? launch_dim<__nv_bfloat16>(a, ws, s) : launch_dim<float>(a, ws, s);
}

}  // namespace ssd
