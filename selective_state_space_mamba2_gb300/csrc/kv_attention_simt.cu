// kv_tree_attention on the CUDA cores, in fp32: every type, head size, group and page size the
// tensor-core kernel does not take, and the kernel that joins the parts of cut items.
//
// Online softmax over key tiles of 32 for 16 query rows a CTA.  Keys and values of a tile come into
// shared memory by 16-byte asynchronous copies, one tile ahead, in their own type.  What bounds such a
// kernel is the reads of shared memory (a 16-byte read of a warp takes 4 cycles whatever is shared in
// it), so a thread takes 4 rows by 4 keys of the scores, each warp a quarter of headdim, and 4 rows by
// 4 columns in 32 of the output, each warp a quarter of the keys: 8 reads for 64 multiply-adds, and 3
// for 32 (a row's scores by one thread took 5 for 16: 37 us for 16 fp32 requests of up to 7 tokens
// and 2000 cached ones, against 28 with this).  The warps' quarters are added up in shared
// memory, the scores' per tile, the output's per item.
#include "kv_sched.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kRowTile = 16;
constexpr int kKeyShift = 5;
constexpr int kKeyTile = 1 << kKeyShift;
constexpr int kOverhead = 1;  // of an item, in key tiles
constexpr int ctas_per_sm(int nv) { return nv <= 2 ? 4 : nv <= 4 ? 3 : 2; }  // by registers
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kStages = 2;
constexpr int kKeyPitch = kRowTile + 4;  // floats of a key's 16 scores or weights: 8 keys side by side in different banks

// a row of keys or values in shared memory: 16 bytes more than it holds, so that 8 rows read side by
// side lie in different banks
template <typename T> __host__ __device__ constexpr int row_bytes(int D) { return D * (int)sizeof(T) + 16; }

template <typename T> constexpr int smem_bytes(int D) {
    return kRowTile * (D + 4) * 4 + kStages * 2 * kKeyTile * row_bytes<T>(D) + 5 * kKeyTile * kKeyPitch * 4;
}

__device__ __forceinline__ float4 get4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 get4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// 16 bytes to shared memory, zeros where `there` is false (src is not read then)
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// NV: 32-float pieces of a row a thread group covers, headdim <= 32 NV
template <typename T, int NV>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NV))
    kv_attention_simt_kernel(const kv_attention_args a, const kvs::Parts parts, const kvs::Tiling g) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ kvs::FindSmem find;
    __shared__ int64_t at_rows[2][2][kKeyTile];
    const int D = a.headdim, group = a.nheads / a.kv_heads, pitch = D + 4;
    const int rb = row_bytes<T>(D), tile_bytes = kKeyTile * rb;
    float *sq = reinterpret_cast<float *>(smem);
    uint8_t *ring = smem + kRowTile * pitch * 4;  // per stage: keys, then values
    float *sp = reinterpret_cast<float *>(ring + kStages * 2 * tile_bytes);  // weights [key][row]
    float *ss = sp + kKeyTile * kKeyPitch;                                    // scores' quarters [warp][key][row]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = tid >> 3, sub = tid & 7;           // softmax and output: a row's eighth
    const int rg = (lane >> 3) * 4, cg = lane & 7;     // products: 4 rows, and keys or columns
    __shared__ __align__(16) float shrinks[kRowTile];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join kernel may be set up
    kvs::Walk w;
    if (!kvs::find_run(a, g, blockIdx.x, gridDim.x, find, parts.borders, w)) return;
    const float c = a.scale * kLog2e;
    constexpr int kPer = 16 / (int)sizeof(T);  // entries of 16 bytes
    const int pieces = D / kPer;
    // Where tile t's keys and values are, in elements from their array's start (-1: nowhere, zeros): found
    // by one warp a tile ahead of the copies, so that these wait for no table entry and divide nothing.
    auto find_rows = [&](int t) {
        const bool cached = t < w.cached_tiles;
        const int32_t pos = (cached ? t : t - w.cached_tiles) * kKeyTile + tid;
        int64_t k_at = -1, v_at = -1;
        if (cached && pos < w.q.c) {
            const int32_t col = pos / a.block_size;
            const int32_t id = a.block_table[(int64_t)w.r * a.table_cols + col];
            if (id >= 0 && id < a.num_blocks)
                k_at = v_at = (int64_t)id * a.cache_block_stride +
                              ((int64_t)(pos - col * a.block_size) * a.kv_heads + w.h) * D;
            else
                report(a.err_word, SSD_DEVERR_SLOT);
        } else if (!cached && pos < w.new_seen) {
            k_at = (int64_t)(w.q.q0 + pos) * a.k_stride + w.h * D;
            v_at = (int64_t)(w.q.q0 + pos) * a.v_stride + w.h * D;
        }
        at_rows[t & 1][0][tid] = k_at;
        at_rows[t & 1][1][tid] = v_at;
    };
    const int key0 = tid / pieces, piece0 = tid - key0 * pieces, key_step = kThreads / pieces,
              piece_step = kThreads - key_step * pieces;
    // The copies of key tile t of the current item into stage `st`.
    auto load = [&](int t, int st) {
        const bool cached = t < w.cached_tiles;
        const T *kp = static_cast<const T *>(cached ? a.k_cache : a.k_new);
        const T *vp = static_cast<const T *>(cached ? a.v_cache : a.v_new);
        uint8_t *k_to = ring + st * 2 * tile_bytes, *v_to = k_to + tile_bytes;
        int piece = piece0;
        for (int key = key0; key < kKeyTile; key += key_step) {
            const int64_t k_at = at_rows[t & 1][0][key], v_at = at_rows[t & 1][1][key];
            const bool there = k_at >= 0;
            copy16(k_to + key * rb + piece * 16, kp + (there ? k_at + piece * kPer : 0), there);
            copy16(v_to + key * rb + piece * 16, vp + (there ? v_at + piece * kPer : 0), there);
            piece += piece_step;
            if (piece >= pieces) piece -= pieces, ++key;
        }
        copies_commit();
    };
    bool more = true;
    while (more) {
        const int heads = w.heads(g, group), rows = w.tokens(g) * heads, head0 = w.h * group + w.part * g.heads;
        const int token0 = w.first_token(g);
        __syncthreads();  // the last item's readers are done
        if (tid < kKeyTile) {
            find_rows(w.t0);
            if (w.t0 + 1 < w.t1) find_rows(w.t0 + 1);
        }
        __syncthreads();
        load(w.t0, 0);
        // query rows
        for (int i = tid; i < kRowTile * (D / 4); i += kThreads) {
            const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int64_t tok = w.q.q0 + token0 + r / heads;
                f = get4(static_cast<const T *>(a.q) + tok * a.q_stride + (head0 + r % heads) * D + e);
            }
            *reinterpret_cast<float4 *>(sq + r * pitch + e) = f;
        }
        const int32_t my_tok = row < rows ? token0 + row / heads : -1;
        const uint32_t *mask = a.tree_mask && my_tok >= 0 ? a.tree_mask + (int64_t)(w.q.q0 + my_tok) * a.mask_words : nullptr;

        float top = -INFINITY, sum = 0.f;
        float2 acc[4][NV][2] = {};
        for (int t = w.t0; t < w.t1; ++t) {
            const bool cached = t < w.cached_tiles;
            const int32_t base = (cached ? t : t - w.cached_tiles) * kKeyTile;
            const int32_t limit = cached ? w.q.c : w.new_seen;  // keys from here on do not exist
            const int st = (t - w.t0) & 1;
            copies_wait<0>();
            __syncthreads();  // tile t is there, and nobody reads the other stage or the last weights any more
            if (t + 1 < w.t1) load(t + 1, st ^ 1);
            if (t + 2 < w.t1 && tid < kKeyTile) find_rows(t + 2);
            const uint8_t *sk = ring + st * 2 * tile_bytes, *sv = sk + tile_bytes;
            // scores of rows rg .. rg + 3 and keys cg + 8 j over this warp's entries, even and odd ones apart
            float2 s2[4][4] = {};
#pragma unroll 2
            for (int e = 4 * warp; e < D; e += 16) {
                float4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sq + (rg + i) * pitch + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 y = get4(reinterpret_cast<const T *>(sk + (cg + 8 * j) * rb) + e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s2[i][j] = tc::fma_f2(make_float2(x[i].x, x[i].y), make_float2(y.x, y.y), s2[i][j]);
                        s2[i][j] = tc::fma_f2(make_float2(x[i].z, x[i].w), make_float2(y.z, y.w), s2[i][j]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4 *>(ss + (warp * kKeyTile + cg + 8 * j) * kKeyPitch + rg) =
                    make_float4(s2[0][j].x + s2[0][j].y, s2[1][j].x + s2[1][j].y, s2[2][j].x + s2[2][j].y,
                                s2[3][j].x + s2[3][j].y);
            __syncthreads();
            // softmax of row `row`, keys sub + 8 j
            float s[4], best = -INFINITY;
            bool sees[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *q4 = ss + (sub + 8 * j) * kKeyPitch + row;
                constexpr int kQuarter = kKeyTile * kKeyPitch;
                s[j] = (q4[0] + q4[kQuarter]) + (q4[2 * kQuarter] + q4[3 * kQuarter]);
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
            if (sub == 0) shrinks[row] = shrink;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // -1 marks what is not seen: a weight may be 0 by underflow, and its value counts all the same
                const float p = sees[j] ? exp2f(s[j] - from) : 0.f;
                sp[(sub + 8 * j) * kKeyPitch + row] = sees[j] ? p : -1.f;
                sum += p;
            }
            __syncthreads();
            // output of rows rg .. rg + 3, columns 32 v + 4 cg, over this warp's keys
            const float4 f4 = *reinterpret_cast<const float4 *>(shrinks + rg);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][v][j] = tc::mul_f2(acc[i][v][j], make_float2(f[i], f[i]));
            const bool all = cached && base + kKeyTile <= limit;  // every row of the item sees every key
#pragma unroll 2
            for (int k = 0; k < kKeyTile / 4; ++k) {
                const int key = warp * (kKeyTile / 4) + k;
                const float4 p4 = *reinterpret_cast<const float4 *>(sp + key * kKeyPitch + rg);
                const float pk[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int e = 32 * v + 4 * cg;
                    const float4 y = e < D ? get4(reinterpret_cast<const T *>(sv + key * rb) + e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p2 = make_float2(pk[i], pk[i]);
                        if (all || !(pk[i] < 0.f)) {  // not seen: its value stays out, whatever it is
                            acc[i][v][0] = tc::fma_f2(p2, make_float2(y.x, y.y), acc[i][v][0]);
                            acc[i][v][1] = tc::fma_f2(p2, make_float2(y.z, y.w), acc[i][v][1]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        // the warps' quarters of the output, over the ring (no copy is in flight): [warp][row][D]
        float *quarters = reinterpret_cast<float *>(ring);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = 32 * v + 4 * cg;
                if (e < D)
                    *reinterpret_cast<float4 *>(quarters + (warp * kRowTile + rg + i) * D + e) =
                        make_float4(acc[i][v][0].x, acc[i][v][0].y, acc[i][v][1].x, acc[i][v][1].y);
            }
        __syncthreads();
        if (my_tok >= 0) {
            const bool whole = w.whole();
            const int64_t out_row = (int64_t)(w.q.q0 + my_tok) * a.nheads + head0 + row % heads;
            const int64_t part = ((int64_t)blockIdx.x * 2 + (w.t0 > 0 ? 0 : 1)) * g.rows + row;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw nothing: zeros
            T *out = static_cast<T *>(a.out) + out_row * D;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = 32 * v + 4 * sub;
                if (e >= D) continue;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 x = *reinterpret_cast<const float4 *>(quarters + (k * kRowTile + row) * D + e);
                    o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                }
                if (whole) {
                    out[e] = from_f32<T>(o.x * inv), out[e + 1] = from_f32<T>(o.y * inv);
                    out[e + 2] = from_f32<T>(o.z * inv), out[e + 3] = from_f32<T>(o.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(parts.sums + part * D + e) = o;
                }
            }
            if (sub == 0) {
                if (!whole)
                    parts.stats[part] = make_float2(top, sum);
                else if (a.lse)
                    a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
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
// A warp sums a row.  Bound by the latency of dependent reads, border, statistics and sums, so the first sums
// are read while the statistics are on their way; for prompts by instructions, hence a short form for few parts
// (trees 178 to 176 us), and the bytes of the parts in L2 (four rows a
// warp: the same).  In tiles of few rows (decode) an item may be in dozens of parts (65536 keys of one
// request: 38): the CTA's four warps then share a row's.
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kAloneParts = 4;   // items of at most so many parts have a warp a row there, too (16 fp32 requests of
                                 // up to 2000 keys 29.2 us, 30.5 with up to 8; one of 777 14.3 us with up to 16)

template <typename T, int NV, bool kFew>  // NV: 128-float pieces of a row
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const kv_attention_args a, const kvs::Parts parts,
                                                               const kvs::Tiling g) {
    __shared__ float4 quarters[kFew ? kJoinWarps : 1][NV * 32];
    const int D = a.headdim, b = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are complete
    const kvs::Border me = parts.borders[b];
    const int n = me.parts, rows = me.tokens * me.heads;
    // CTAs of tiles of few rows: every fourth one has four rows, or each has one
    const bool alone = !kFew || n <= kAloneParts;
    const int row = kFew ? blockIdx.y + (alone ? warp : 0) : blockIdx.y * kJoinWarps + warp;
    if (n == 0 || row >= rows || (kFew && alone && blockIdx.y % kJoinWarps != 0)) return;
    // part k: of CTA b - 1 + k
    auto part_row = [&](int k) { return ((int64_t)(b - 1 + k) * 2 + (k == 0 ? 1 : 0)) * g.rows + row; };
    float top = -INFINITY, sum = 0.f;
    float4 acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto read = [&](int k, float4 (&v)[NV]) {
        const float *src = parts.sums + part_row(k) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            v[j] = 128 * j + 4 * lane < D ? *reinterpret_cast<const float4 *>(src + 128 * j + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto add = [&](float f, const float4 (&v)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            acc[j].x = fmaf(f, v[j].x, acc[j].x);
            acc[j].y = fmaf(f, v[j].y, acc[j].y);
            acc[j].z = fmaf(f, v[j].z, acc[j].z);
            acc[j].w = fmaf(f, v[j].w, acc[j].w);
        }
    };
    if (!kFew && n <= kAloneParts) {  // every lane has all statistics: with many rows the instructions count
        float4 v[kAloneParts][NV];
        float2 st[kAloneParts];
#pragma unroll
        for (int k = 0; k < kAloneParts; ++k) {
            if (k >= n) break;
            read(k, v[k]);
            st[k] = parts.stats[part_row(k)];
        }
#pragma unroll
        for (int k = 0; k < kAloneParts; ++k) {
            if (k >= n) break;
            top = st[k].x > top || st[k].x != st[k].x ? st[k].x : top;
        }
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < kAloneParts; ++k) {
            if (k >= n) break;
            const float f = exp2f(st[k].x - from);
            sum = fmaf(f, st[k].y, sum);
            add(f, v[k]);
        }
    } else {
        constexpr int kFlight = 4;  // parts in flight
        const int share = alone ? 0 : warp, step = alone ? 1 : kJoinWarps;  // parts of this warp
        float4 v[kFlight][NV];
        auto read_some = [&](int k) {  // the last ones repeated
#pragma unroll
            for (int i = 0; i < kFlight; ++i) read(k + i * step < n ? k + i * step : k, v[i]);
        };
        if (share < n) read_some(share);
        float2 st = lane < n ? parts.stats[part_row(lane)] : make_float2(-INFINITY, 0.f);  // a lane a part
        top = st.x;
        for (int k = lane + 32; k < n; k += 32) {
            const float m = parts.stats[part_row(k)].x;
            top = m > top || m != m ? m : top;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m = __shfl_xor_sync(~0u, top, o);
            top = m > top || m != m ? m : top;
        }
        const float from = top == -INFINITY ? 0.f : top;
        for (int k0 = 0; k0 < n; k0 += 32) {
            if (k0 > 0) st = k0 + lane < n ? parts.stats[part_row(k0 + lane)] : make_float2(-INFINITY, 0.f);
            const float f = k0 + lane < n ? exp2f(st.x - from) : 0.f;
            sum = fmaf(f, st.y, sum);
            for (int k = k0 + share; k < min(n, k0 + 32); k += kFlight * step) {
                if (k > share) read_some(k);
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const float fk = __shfl_sync(~0u, f, (k + i * step) & 31);
                    if (k + i * step < n) add(fk, v[i]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (!alone) {
#pragma unroll
            for (int j = 0; j < NV; ++j) quarters[warp][j * 32 + lane] = acc[j];
            __syncthreads();
            if (warp > 0) return;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) {
                    const float4 q = quarters[w][j * 32 + lane];
                    acc[j].x += q.x, acc[j].y += q.y, acc[j].z += q.z, acc[j].w += q.w;
                }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row that saw nothing: zeros
    const int64_t out_row = (int64_t)(me.token0 + row / me.heads) * a.nheads + me.head0 + row % me.heads;
    T *out = static_cast<T *>(a.out) + out_row * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = 128 * j + 4 * lane;
        if (e >= D) continue;
        const float4 o = make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4 *>(out + e) = o;
        else
            *reinterpret_cast<uint2 *>(out + e) = make_uint2(tc::pack_bf16(o.x, o.y), tc::pack_bf16(o.z, o.w));
    }
    if (a.lse && lane == 0) a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <typename T, int NV>
cudaError_t launch_join(const kv_attention_args &a, const kvs::Parts &p, int grid, const kvs::Tiling &g, cudaStream_t s) {
    // a programmatic dependent of the attention kernel: its CTAs may be set up while that ends
    const bool few = g.rows <= kvs::kFewRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)(few ? g.rows : kvs::ceil_div(g.rows, kJoinWarps)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, kv_join_kernel<T, NV, true>, a, p, g)
               : cudaLaunchKernelEx(&cfg, kv_join_kernel<T, NV, false>, a, p, g);
}

kvs::Tiling simt_tiling(const kv_attention_args &a) { return kvs::tiling(a, kRowTile, kKeyShift, kOverhead, 1); }

// 32-float pieces of a row that the kernel for this head size covers
int pieces_of(int D) { return D <= 64 ? 2 : D <= 128 ? 4 : 8; }

int smem_of(const kv_attention_args &a) {
    return a.dtype == SSD_BF16 ? smem_bytes<__nv_bfloat16>(a.headdim) : smem_bytes<float>(a.headdim);
}

int simt_grid(const kv_attention_args &a, const kvs::Tiling &g) {
    const int by_smem = (227 * 1024) / (smem_of(a) + 3 * 1024);  // with what a CTA takes besides
    const int ctas = ctas_per_sm(pieces_of(a.headdim));
    return kvs::grid_of(a, g, (by_smem < ctas ? by_smem : ctas) * device_sms());
}

template <typename T, int NV>
cudaError_t launch(const kv_attention_args &a, void *ws, cudaStream_t s) {
    const kvs::Tiling g = simt_tiling(a);
    const int grid = simt_grid(a, g);
    const kvs::Parts parts = kvs::parts_at(ws, grid, g.rows, a.headdim);
    const int smem = smem_of(a);
    cudaError_t e = cudaFuncSetAttribute(kv_attention_simt_kernel<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kv_attention_simt_kernel<T, NV><<<grid, kThreads, smem, s>>>(a, parts, g);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kvs::join_launch(a, parts, grid, g, s);
}

template <typename T> cudaError_t launch_dim(const kv_attention_args &a, void *ws, cudaStream_t s) {
    const int pieces = pieces_of(a.headdim);
    return pieces == 2 ? launch<T, 2>(a, ws, s) : pieces == 4 ? launch<T, 4>(a, ws, s) : launch<T, 8>(a, ws, s);
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
