// gdn_rope.cu -- what a full-attention layer of a hybrid stack does to its new tokens'
// projections before attention: RMS norm of every query and key head, the position
// rotation, and the append of the keys and values to a paged cache, in one pass.
//
// Per row r (position p) and head, x in R^d:
//   y = x rsqrt(mean(x^2) + eps) w           (no weight: y = x)
//   pair (a, b) of the first rotary_dim elements, frequency f_i:
//   (a, b) -> (a cos(p f_i) - b sin(p f_i), b cos(p f_i) + a sin(p f_i))
// Per element that is (x A + x' B) r with x' the pair's other element, A = w cos,
// B = -+ w' sin and r the head's inverse root: A and B are constants of a row, kept in
// registers while a lane walks its heads.
//
// Every element is read once and written once with about 7 flops in between, so HBM
// bounds it.  16 bytes per lane: one head is 8 to 32 lanes, the sum of squares a
// shuffle tree over them in fp32, x' (split halves) one shuffle of the raw 16 bytes.
// Four heads are loaded ahead, the first four before the angles are computed: the
// 67001-row case (24 heads of 128, bf16, 824 MB) takes 146 us so, 5.7 TB/s, and took 213,
// 170 and 172 us with one, two and eight.  The result is rounded once, from fp32, when it
// is stored.
//
// The angle holds for far positions without a table and without fp64 per pair: a
// turn is 2^64, so p f_i mod 2 pi is the low 64 bits of p times the frequency in turns
// as a 64-bit fraction, one integer product that wraps by itself.  The fraction comes
// from the fp64 frequency (error below 2^-52 of f, and 2^-64 of a turn where it is cut off;
// both times p), its signed value is rounded to fp32 (2^-24 of a half turn, which hides them
// up to p = 2^28) and goes to sincospif.  A block computes the cosines and sines
// of its rows once, in shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_f32x2.h"
#include "gdn_hybrid.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

constexpr int kAhead = 4;   // heads loaded ahead

template <typename T>
struct Vec16;   // 16 bytes of T as fp32 values
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    __device__ static void unpack(uint4 x, float* v) {
        v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    }
    __device__ static uint4 pack(const float* v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(uint4 x, float* v) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float* v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Block: RT consecutive rows (blockIdx.x) and the heads of one of gridDim.y shares; the
// lane groups are dealt to the rows, and each walks its row's share of the q heads, then of
// the k heads, then of the v heads, each with a loop of its own: with one loop that asked
// for every head which of them it was, a warp issued 181 instructions for its two heads
// instead of 114 and the 67001-row case was bound by that (174 us).
template <typename T, int D, int RT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const NormRopeArgs a) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    constexpr int LPH = D / N;                  // lanes of one head
    constexpr int GROUPS = kThreads / LPH;      // heads in flight in the block
    static_assert(GROUPS % RT == 0, "every row gets the same number of lane groups");
    static_assert(RT == 1 || RT >= 32 / LPH, "the lane groups of a warp walk the same heads, of different rows");
    constexpr int GPR = GROUPS / RT;            // lane groups of one row
    __shared__ float2 cs[RT][D / 2];

    const long long row_base = (long long)blockIdx.x * RT;
    const int group = threadIdx.x / LPH, l = threadIdx.x % LPH, lane = threadIdx.x & 31;
    const unsigned lanes = RT > 1 || LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1) << (lane - l);   // that walk as this one
    const int rl = group % RT;
    const long long row = row_base + rl;
    const bool row_ok = row < a.rows;
    const int e0 = l * N;                       // first element of this lane

    // this lane's heads: every step-th of q, k and (with a cache) v heads in a row, so that few
    // rows spread their heads evenly
    const int Hq = a.num_heads, Hkv = a.num_kv_heads;
    const int step = GPR * gridDim.y;
    auto first_from = [&](int h, int count) {   // in the list after one of `count` heads entered at h
        return h >= count ? h - count : h + (count - h + step - 1) / step * step - count;
    };
    const int hq = group / RT + GPR * blockIdx.y;
    const int hk = first_from(hq, Hq);
    const int hv = first_from(hk, Hkv);
    const T* q = static_cast<const T*>(a.q) + row * a.rs_q + e0;
    const T* k = static_cast<const T*>(a.k) + row * a.rs_k + e0;
    const T* v = static_cast<const T*>(a.v) + row * a.rs_v + e0;
    uint4 raw[kAhead];
    auto load = [&](const T* list, int h, int count) {
        const T* from = list + (long long)h * D;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row_ok && h + i * step < count) raw[i] = *reinterpret_cast<const uint4*>(from);
            from += (long long)step * D;
        }
    };
    if (hq < Hq) load(q, hq, Hq);
    else if (hk < Hkv) load(k, hk, Hkv);
    T* k_page = nullptr;
    T* v_page = nullptr;
    if (row_ok && a.slots) {
        const long long slot = a.slots[row];
        if (slot >= 0 && slot < (long long)a.num_pages * a.page_size) {
            const long long page = slot <= 0xffffffffll ? (uint32_t)slot / (uint32_t)a.page_size : slot / a.page_size;
            const long long off = page * a.page_stride + (slot - page * a.page_size) * a.cache_row_stride + e0;
            k_page = static_cast<T*>(a.k_pages) + off;
            v_page = static_cast<T*>(a.v_pages) + off;
        }
    }

    const int half = a.rotary_dim / 2;
    // a thread per frequency, and as many sets of them over the rows as the block has room for
    const int sets = half > 0 ? kThreads / half : 0;
    if ((int)threadIdx.x < sets * half) {
        const int j = threadIdx.x % half;
        double f = a.inv_freq[j] * 0.15915494309189533577;   // 1 / (2 pi): turns per position
        f -= floor(f);
        const unsigned long long turn = __double2ull_rz(f * 18446744073709551616.0);   // 2^64
        for (int r = threadIdx.x / half; r < RT && row_base + r < a.rows; r += sets) {
            const unsigned long long at = (unsigned long long)a.positions[row_base + r] * turn;
            float sn, c;
            sincospif(__ll2float_rn((long long)at) * 1.0842021724855044e-19f, &sn, &c);   // 2^-63: half turns
            cs[r][j] = make_float2(c, sn);
        }
    }
    __syncthreads();

    const bool rot = e0 < a.rotary_dim;
    // the lane of the pair's other half (split halves); half is a multiple of N
    const bool upper = e0 >= half;
    const int partner = !rot ? lane : lane - l + (upper ? l - half / N : l + half / N);
    const int pe0 = INTERLEAVED || !rot ? e0 : upper ? e0 - half : e0 + half;   // its first element

    // norm and rotation of this lane's heads of one list; `store` gets each with its number
    auto walk = [&](const T* list, int h, int count, const float* w, bool loaded, auto store) {
        if (h >= count) return;
        Pair A[N / 2], B[N / 2];
        float wo[N], wp[N], av[N], bv[N];
#pragma unroll
        for (int i = 0; i < N; ++i) wo[i] = wp[i] = 1.0f;
        if (w) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                *reinterpret_cast<float4*>(wo + i) = *reinterpret_cast<const float4*>(w + e0 + i);
                *reinterpret_cast<float4*>(wp + i) = *reinterpret_cast<const float4*>(w + pe0 + i);
            }
        }
        const int c0 = INTERLEAVED ? e0 / 2 : upper ? e0 - half : e0;   // this lane's first angle
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 x = rot ? cs[rl][INTERLEAVED ? c0 + i / 2 : c0 + i] : make_float2(1.0f, 0.0f);
            const bool first = INTERLEAVED ? i % 2 == 0 : !upper;   // a pair's first element: minus
            av[i] = wo[i] * x.x;
            bv[i] = wp[INTERLEAVED ? i ^ 1 : i] * (first ? -x.y : x.y);
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            A[i] = pair(av[2 * i], av[2 * i + 1]);
            B[i] = pair(bv[2 * i], bv[2 * i + 1]);
        }
        for (; h < count; h += kAhead * step, loaded = false) {
            if (!loaded) load(list, h, count);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int head = h + u * step;
                if (head >= count) break;
                float xs[N];
                V::unpack(raw[u], xs);
                Pair x[N / 2], sq = pair(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    x[i] = pair(xs[2 * i], xs[2 * i + 1]);
                    sq = fma2(x[i], x[i], sq);
                }
                const float2 sums = unpair(sq);
                float ss = sums.x + sums.y;
#pragma unroll
                for (int m = LPH / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(lanes, ss, m);
                const float r = w ? rsqrtf(ss * (1.0f / D) + a.eps) : 1.0f;
                float os[N];
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int i = 0; i < N; ++i) os[i] = xs[i ^ 1];
                } else {
                    uint4 other;
                    other.x = __shfl_sync(lanes, raw[u].x, partner);
                    other.y = __shfl_sync(lanes, raw[u].y, partner);
                    other.z = __shfl_sync(lanes, raw[u].z, partner);
                    other.w = __shfl_sync(lanes, raw[u].w, partner);
                    V::unpack(other, os);
                }
                // x A before r: an x whose square is finite is far from overflowing there
                const Pair rr = pair(r, r);
                float z[N];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    Pair t = mul2(x[i], A[i]);
                    if (rot) t = fma2(pair(os[2 * i], os[2 * i + 1]), B[i], t);
                    const float2 y = unpair(mul2(t, rr));
                    z[2 * i] = y.x;
                    z[2 * i + 1] = y.y;
                }
                if (row_ok) store(head, V::pack(z));
            }
        }
    };
    T* q_out = static_cast<T*>(a.q_out) + row * Hq * D + e0;
    walk(q, hq, Hq, a.q_weight, true, [&](int h, uint4 out) { *reinterpret_cast<uint4*>(q_out + h * D) = out; });
    T* k_out = a.k_out ? static_cast<T*>(a.k_out) + row * Hkv * D + e0 : nullptr;
    walk(k, hk, Hkv, a.k_weight, hq >= Hq, [&](int h, uint4 out) {
        if (k_out) *reinterpret_cast<uint4*>(k_out + h * D) = out;
        if (k_page) *reinterpret_cast<uint4*>(k_page + h * a.cache_head_stride) = out;
    });
    if (!a.slots) return;
    for (int h = hv; h < Hkv; h += kAhead * step) {   // the values go in as they came
        load(v, h, Hkv);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (v_page && h + u * step < Hkv)
                *reinterpret_cast<uint4*>(v_page + (h + u * step) * a.cache_head_stride) = raw[u];
    }
}

template <typename T, int D, int RT, bool IL>
cudaError_t launch_rt(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int GPR = kThreads / (D / Vec16<T>::N) / RT;
    const int heads = a.num_heads + (a.slots ? 2 : 1) * a.num_kv_heads;
    const long long row_tiles = (a.rows + RT - 1) / RT;
    // few rows: their heads spread over more blocks, down to one head per lane group, until
    // the grid has about two blocks per SM
    const long long most = (heads + GPR - 1) / GPR;
    const long long shares = std::max(1ll, std::min(most, (296 + row_tiles - 1) / row_tiles));
    norm_rope_kernel<T, D, RT, IL><<<dim3((unsigned)row_tiles, (unsigned)shares), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// One row per block while the rows are few, so that a row's heads spread over all lane
// groups; eight rows per block otherwise, and one per lane group (at most 16) once that
// still gives two blocks per SM: A and B then last for all heads of a row (67001 rows of 24
// heads: 234, 174 and 146 us with 4, 8 and 16 rows; 1024 rows of 96: 18 us with each).
template <typename T, int D, bool IL>
cudaError_t launch_rows(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int GROUPS = kThreads / (D / Vec16<T>::N);
    constexpr int MANY = GROUPS < 16 ? GROUPS : 16;
    if (a.rows <= 296) return launch_rt<T, D, 1, IL>(a, stream);
    return a.rows < 296 * MANY ? launch_rt<T, D, 8, IL>(a, stream) : launch_rt<T, D, MANY, IL>(a, stream);
}

template <typename T, int D>
cudaError_t launch_style(const NormRopeArgs& a, cudaStream_t stream) {
    return a.interleaved ? launch_rows<T, D, true>(a, stream) : launch_rows<T, D, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    if (a.dtype == GDN_F32)
        return a.dim == 64 ? launch_style<float, 64>(a, stream) : launch_style<float, 128>(a, stream);
    return a.dim == 64 ? launch_style<__nv_bfloat16, 64>(a, stream) : launch_style<__nv_bfloat16, 128>(a, stream);
}

}  // namespace gdn
