// gdn_attn.cu -- attention of a chunk of new tokens over a paged cache: the kernels that
// lay out and merge the work (gdn_attn.h), and the fp32 attention kernel.
//
// Per new token i of a sequence with n new tokens and context L (position p = L - n + i)
// and query head h, over the keys j in (p - window, p], j >= 0, of key head h / group:
//   o = sum_j softmax_j(scale q . k_j) v_j,    lse = log sum_j exp(scale q . k_j)
// in one pass over the keys with a running maximum and sum.  A row without keys gives
// o = 0 and lse = -infinity.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "gdn_attn.h"

namespace gdn {
namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ the line
// One block.  A warp per sequence sums the tiles of its token blocks; a scan over the
// sequences places them on the line.  A sequence whose entries do not fit the call's
// extents gets no work (its rows stay as they were) and the status says so.
__global__ void __launch_bounds__(1024) line_kernel(const Args a) {
    __shared__ long long warp_sum[32];
    __shared__ long long carry;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        a.ws->epoch = a.epoch;
        carry = 0;
    }
    const long long max_ctx = (long long)a.max_pages * a.page_size;
    for (int b = warp; b < a.batch; b += 32) {
        const int r0 = a.cu[b], r1 = a.cu[b + 1], ctx = a.ctx[b];
        const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.rows && ctx >= 0 && ctx <= max_ctx;
        Seq s;
        s.row0 = r0;
        s.qlen = good ? r1 - r0 : 0;
        s.ctx = ctx;
        s.pad = 0;
        long long n = 0;
        const int blocks = token_blocks(a, s.qlen);
        for (int t = lane; t < blocks; t += 32) n += block_range(a, s.qlen, ctx, t).tiles;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        s.head_tiles = n;
        s.before = 0;
        if (lane == 0) {
            a.seqs[b] = s;
            if (!good) report(a, kStatusMismatch);
        }
    }
    __syncthreads();
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        const long long n = b < a.batch ? a.seqs[b].head_tiles * a.num_kv_heads : 0;
        long long incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            long long w = warp_sum[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, w, d);
                if (lane >= d) w += x;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        const long long before = carry + (warp ? warp_sum[warp - 1] : 0) + incl - n;
        if (b < a.batch) a.seqs[b].before = before;
        __syncthreads();
        if (threadIdx.x == 0) carry += warp_sum[31];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const long long total = carry;
        long long per = (total + a.shape.max_parts - 1) / a.shape.max_parts;
        if (per < a.shape.min_tiles) per = a.shape.min_tiles;
        a.line->total = total;
        a.line->per_part = per;
        a.line->parts = (int)((total + per - 1) / per);
    }
}

// --------------------------------------------------------------- the merge
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 x);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 x) {
    *reinterpret_cast<float4*>(p) = x;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 x) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Block (i, y): the unit that the cut before CTA i + 1 is the first to split, rows
// 8 y .. 8 y + 7, a warp per row.  Weights exp2(lse - max) over the unit's parts, in the
// order of the line.  Bound by latency: a few hundred KB at most.
template <typename T>
__global__ void __launch_bounds__(256) combine_kernel(const Args a) {
    const long long part = (long long)blockIdx.x + 1;
    const Line& ln = *a.line;
    if (part >= ln.parts) return;
    const long long per = ln.per_part, cut = part * per;
    const Unit u = find_unit(a, cut);
    if (u.begin == cut) return;                    // a unit begins here: nothing is split
    const long long first = u.begin / per, last = (u.begin + u.r.tiles - 1) / per;
    if (first != part - 1) return;                 // an earlier cut's block merges it
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int unit_rows = a.shape.subs * a.shape.sub_rows;
    if (row >= unit_rows) return;
    const int in = row % a.shape.sub_rows;
    const int tok = (row / a.shape.sub_rows) * a.block_tokens + in / a.group;
    if (in >= a.block_tokens * a.group || tok >= u.r.toks) return;

    auto slot_row = [&](long long p) {
        const bool begins = p > first || u.begin == first * per;
        return part_slot(p, begins) * unit_rows + row;
    };
    float top = -INFINITY;
    for (long long p = first + lane; p <= last; p += 32) top = fmaxf(top, a.part_lse[slot_row(p)]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float ref = top == -INFINITY ? 0.0f : top;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    const bool mine = lane * 4 < a.dim;
#pragma unroll 4
    for (long long p = first; p <= last; ++p) {
        const long long sr = slot_row(p);
        const float w = exp2f(a.part_lse[sr] - ref);
        sum += w;
        if (mine && w > 0.0f) {
            const float4 x = *reinterpret_cast<const float4*>(a.part_o + sr * a.dim + lane * 4);
            acc.x = fmaf(w, x.x, acc.x);
            acc.y = fmaf(w, x.y, acc.y);
            acc.z = fmaf(w, x.z, acc.z);
            acc.w = fmaf(w, x.w, acc.w);
        }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const long long orow = (long long)(u.s.row0 + u.r.tok0 + tok) * a.num_heads + u.head * a.group + in % a.group;
    if (mine)
        store4(static_cast<T*>(a.o) + orow * a.dim + lane * 4,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0) a.lse[orow] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------- fp32 attention
// 64 rows x 64 keys per tile on the CUDA cores.  256 threads: thread (ty, tx) holds the
// scores of rows 4 ty .. 4 ty + 3 and keys tx + 16 j, and the outputs of those rows and
// columns 4 tx + 64 j.  K and V of a tile take turns in one shared buffer, so that two
// CTAs share an SM.  Bound by the fp32 pipe (4 d flops per row and key).
constexpr int kRows = 64, kKeys = 64, kThreads = 256;

template <int D>
struct SimtSmem {
    static constexpr int LD = D + 4;               // padded row: float4 reads of 8 rows hit 32 banks
    float q[kRows][LD];
    float kv[kKeys][LD];
    float p[kRows][kKeys + 4];
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
__global__ void __launch_bounds__(kThreads, 2) simt_kernel(const Args a) {
    extern __shared__ float smem_raw[];
    SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem_raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const long long per = a.line->per_part;
    if ((int)blockIdx.x >= a.line->parts) return;
    long long pos = (long long)blockIdx.x * per;
    const long long end = min(pos + per, a.line->total);
    Unit u = find_unit(a, pos);
    const float scale = a.scale * kLog2e;
    bool begins = true;
    while (pos < end) {
        const int kt0 = (int)(pos - u.begin);
        const int kt1 = (int)min((long long)u.r.tiles, end - u.begin);
        const int rows = u.r.toks * a.group;
        const int first_pos = u.s.ctx - u.s.qlen + u.r.tok0;
        // queries
        for (int i = tid; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows)
                x = load4(static_cast<const float*>(a.q) + (long long)(u.s.row0 + u.r.tok0 + r / a.group) * a.rs_q +
                          (long long)(u.head * a.group + r % a.group) * D + c);
            *reinterpret_cast<float4*>(&sm.q[r][c]) = x;
        }
        float m[4], l[4], o[4][D / 16];
        int top_key[4], low_key[4];                // keys [low, top] are seen
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
            top_key[i] = first_pos + (4 * ty + i) / a.group;
            low_key[i] = a.window > 0 ? max(0, top_key[i] - a.window + 1) : 0;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] = 0.0f;
        }
        // this tile's K (or V) rows, zero outside the unit's keys
        auto load_rows = [&](const void* base, int key0) {
            for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = (i % (D / 4)) * 4;
                const int key = key0 + r;
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (key >= u.r.lo && key < u.r.hi) {
                    const int page = a.page_table[(long long)u.b * a.max_pages + key / a.page_size];
                    if (page >= 0 && page < a.num_pages)
                        x = load4(static_cast<const float*>(base) + (long long)page * a.page_stride +
                                  (long long)(key % a.page_size) * a.row_stride + (long long)u.head * a.head_stride + c);
                    else if (c == 0)
                        report(a, kStatusMismatch);
                }
                *reinterpret_cast<float4*>(&sm.kv[r][c]) = x;
            }
        };
        const bool active = (4 * (ty & ~1)) < rows;   // warp-uniform: some row of this warp is a real one
        for (int kt = kt0; kt < kt1; ++kt) {
            const int key0 = (u.r.tile0 + kt) * kKeys;
            load_rows(a.k, key0);
            __syncthreads();
            float s[4][4];
            if (active) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    float4 qv[4], kv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + i][c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&sm.kv[tx + 16 * j][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                            s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                            s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                            s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float top = m[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = key0 + tx + 16 * j;
                        s[i][j] = key >= low_key[i] && key <= top_key[i] ? s[i][j] * scale : -INFINITY;
                        top = fmaxf(top, s[i][j]);
                    }
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    const float keep = exp2f(m[i] - ref);
                    m[i] = top;
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = exp2f(s[i][j] - ref);
                        sum += s[i][j];
                        sm.p[4 * ty + i][tx + 16 * j] = s[i][j];
                    }
                    l[i] = l[i] * keep + sum;      // this lane's share of the row's sum
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) o[i][j] *= keep;
                }
            }
            __syncthreads();                       // K is read, P is written
            load_rows(a.v, key0);
            __syncthreads();
            if (active) {
#pragma unroll 2
                for (int c = 0; c < kKeys; c += 4) {
                    float4 pv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4*>(&sm.p[4 * ty + i][c]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < D / 64; ++j) {
                            const float4 x = *reinterpret_cast<const float4*>(&sm.kv[c + e][4 * tx + 64 * j]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float p = e == 0 ? pv[i].x : e == 1 ? pv[i].y : e == 2 ? pv[i].z : pv[i].w;
                                o[i][4 * j] = fmaf(p, x.x, o[i][4 * j]);
                                o[i][4 * j + 1] = fmaf(p, x.y, o[i][4 * j + 1]);
                                o[i][4 * j + 2] = fmaf(p, x.z, o[i][4 * j + 2]);
                                o[i][4 * j + 3] = fmaf(p, x.w, o[i][4 * j + 3]);
                            }
                        }
                }
            }
            __syncthreads();                       // V and P are read
        }
        const bool whole = kt0 == 0 && kt1 == u.r.tiles;
        if (active) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float sum = l[i];
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
                const float lse2 = sum > 0.0f ? m[i] + log2f(sum) : -INFINITY;
                const int r = 4 * ty + i;
                if (r >= rows) continue;
                const long long orow = (long long)(u.s.row0 + u.r.tok0 + r / a.group) * a.num_heads +
                                       u.head * a.group + r % a.group;
                const long long prow = part_slot(blockIdx.x, begins) * kRows + r;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const float4 x = make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                                                 o[i][4 * j + 3] * inv);
                    if (whole) store4(static_cast<float*>(a.o) + orow * D + 4 * tx + 64 * j, x);
                    else *reinterpret_cast<float4*>(a.part_o + prow * D + 4 * tx + 64 * j) = x;
                }
                if (tx == 0) {
                    if (whole) {
                        if (a.lse) a.lse[orow] = lse2 * kLn2;
                    } else {
                        a.part_lse[prow] = lse2;
                    }
                }
            }
        }
        pos = u.begin + kt1;
        begins = false;
        if (pos < end) next_unit(a, u);
        __syncthreads();
    }
}

template <int D>
cudaError_t launch_simt_typed(const Args& a, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e =
        ensure_smem_limit(reinterpret_cast<const void*>(simt_kernel<D>), (int)sizeof(SimtSmem<D>), smem_set);
    if (e != cudaSuccess) return e;
    simt_kernel<D><<<a.shape.max_parts, kThreads, sizeof(SimtSmem<D>), stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

constexpr Shape kSimtShape{kRows, 1, kKeys, 296, 2};

cudaError_t launch_simt(const Args& a, cudaStream_t stream) {
    return a.dim == 64 ? launch_simt_typed<64>(a, stream) : launch_simt_typed<128>(a, stream);
}

}  // namespace attn

attn::Shape paged_attention_shape(int dtype, int) { return dtype == GDN_F32 ? attn::kSimtShape : attn::shape_tc(); }

attn::Layout paged_attention_layout(int dtype, int dim, int batch) {
    const attn::Shape sh = paged_attention_shape(dtype, dim);
    const size_t rows = (size_t)2 * sh.max_parts * sh.subs * sh.sub_rows;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    attn::Layout l;
    l.line = sizeof(WorkspaceHeader);
    l.seqs = l.line + sizeof(attn::Line);
    l.part_lse = l.seqs + up(sizeof(attn::Seq) * (size_t)batch);
    l.part_o = l.part_lse + up(sizeof(float) * rows);
    l.bytes = l.part_o + up(sizeof(float) * rows * dim);
    return l;
}

cudaError_t launch_paged_attention(const attn::Args& a, cudaStream_t stream) {
    attn::line_kernel<<<1, 1024, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = a.dtype == GDN_F32 ? attn::launch_simt(a, stream) : attn::launch_tc(a, stream);
    if (e != cudaSuccess) return e;
    // rows of a unit, at most those of the call
    const long long unit_rows = (long long)a.shape.subs * a.shape.sub_rows;
    const long long y = a.rows < a.block_tokens ? a.rows * a.group : unit_rows;
    const dim3 grid((unsigned)(a.shape.max_parts - 1), (unsigned)((y + 7) / 8));
    if (a.dtype == GDN_F32) attn::combine_kernel<float><<<grid, 256, 0, stream>>>(a);
    else attn::combine_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
