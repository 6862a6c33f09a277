// gdn_rope.cu -- what a full-attention layer of a hybrid stack does to its new tokens'
// projections before attention: RMS norm of every query and key head, the position
// rotation, and the append of the keys and values to a paged cache, in one pass.
//
// Per row r (position p) and head, x in R^d:
//   y = x rsqrt(mean(x^2) + eps) w           (no weight: y = x)
//   pair (a, b) of the first rotary_dim elements, frequency f_i:
//   (a, b) -> (a cos(p f_i) - b sin(p f_i), b cos(p f_i) + a sin(p f_i))
//
// Every element is read once and written once with about 7 flops in between, so HBM
// bounds it.  16 bytes per lane: one head is 8 to 32 lanes, the sum of squares a
// shuffle tree over them in fp32, and (split halves) a pair's other element a shuffle
// away.  The result is rounded once, from fp32, when it is stored.
//
// The angle is exact for far positions without a table and without fp64 per pair: a
// turn is 2^64, so p f_i mod 2 pi is the low 64 bits of p times the frequency in turns
// as a 64-bit fraction, one integer product that wraps by itself.  The fraction comes
// from the fp64 frequency (error below 2^-52 of f), its signed value is rounded to fp32
// (2^-24 of a half turn) and goes to sincospif.  A block computes the cosines and sines
// of its rows once, in shared memory; the lanes that share a row keep theirs in
// registers over the row's heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec16;   // 16 bytes of T as fp32 values
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    __device__ static void load(const float* p, float* v) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    }
    __device__ static void store(float* p, const float* v) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void load(const __nv_bfloat16* p, float* v) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static void store(__nv_bfloat16* p, const float* v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Block: RT consecutive rows (blockIdx.x) and the heads of one of gridDim.y shares; the
// lane groups are dealt to the rows, and each walks its row's share of the q, k and v heads.
template <typename T, int D, int RT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
    using V = Vec16<T>;
    constexpr int N = V::N;
    constexpr int LPH = D / N;                  // lanes of one head
    constexpr int GROUPS = kThreads / LPH;      // heads in flight in the block
    static_assert(GROUPS % RT == 0, "every row gets the same number of lane groups");
    constexpr int GPR = GROUPS / RT;            // lane groups of one row
    __shared__ float2 cs[RT][D / 2];

    const long long row_base = (long long)blockIdx.x * RT;
    const int half = a.rotary_dim / 2;
    for (int i = threadIdx.x; i < RT * half; i += kThreads) {
        const int r = i / half, j = i - r * half;
        if (row_base + r < a.rows) {
            double f = a.inv_freq[j] * 0.15915494309189533577;   // 1 / (2 pi): turns per position
            f -= floor(f);
            const unsigned long long turn = __double2ull_rz(f * 18446744073709551616.0);   // 2^64
            const unsigned long long at = (unsigned long long)a.positions[row_base + r] * turn;
            float s, c;
            sincospif(__ll2float_rn((long long)at) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
            cs[r][j] = make_float2(c, s);
        }
    }
    __syncthreads();

    const int group = threadIdx.x / LPH, l = threadIdx.x % LPH;
    const int rl = group % RT;
    const long long row = row_base + rl;
    const bool row_ok = row < a.rows;
    const int e0 = l * N;                       // first element of this lane
    const bool rot = e0 < a.rotary_dim;
    // the lane of the pair's other half (split halves); half is a multiple of N
    const int base_lane = (threadIdx.x & 31) - l;
    const int partner = !rot ? (threadIdx.x & 31) : base_lane + (e0 < half ? l + half / N : l - half / N);
    const bool upper = e0 >= half;
    float c[N], s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = INTERLEAVED ? (e0 + i) / 2 : (upper ? e0 + i - half : e0 + i);
        const float2 x = rot && row_ok ? cs[rl][j] : make_float2(1.0f, 0.0f);
        c[i] = x.x;
        // the sign of the second product: minus for a pair's first element
        const bool first = INTERLEAVED ? (i % 2 == 0) : !upper;
        s[i] = first ? -x.y : x.y;
    }
    T* k_page = nullptr;
    T* v_page = nullptr;
    if (row_ok && a.slots) {
        const long long slot = a.slots[row];
        if (slot >= 0 && slot < (long long)a.num_pages * a.page_size) {
            const long long page = slot / a.page_size, at = slot - page * a.page_size;
            const long long off = page * a.page_stride + at * a.cache_row_stride;
            k_page = static_cast<T*>(a.k_pages) + off;
            v_page = static_cast<T*>(a.v_pages) + off;
        }
    }

    // this block's heads: q heads 0 .. Hq, then k heads, then v heads (cache only)
    const int Hq = a.num_heads, Hkv = a.num_kv_heads;
    const int heads = Hq + (a.slots ? 2 : 1) * Hkv;
    const int step = GPR * gridDim.y;
    const int first_head = group / RT + GPR * blockIdx.y;
    const int rounds = (heads + step - 1) / step;       // the same for every lane: shuffles stay whole
    for (int it = 0; it < rounds; ++it) {
        const int hh = first_head + it * step;
        const bool ok = row_ok && hh < heads;
        const bool is_q = hh < Hq, is_k = !is_q && hh < Hq + Hkv;
        const int h = is_q ? hh : is_k ? hh - Hq : hh - Hq - Hkv;
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.0f;
        if (ok) {
            const T* src = is_q   ? static_cast<const T*>(a.q) + row * a.rs_q
                           : is_k ? static_cast<const T*>(a.k) + row * a.rs_k
                                  : static_cast<const T*>(a.v) + row * a.rs_v;
            V::load(src + (long long)h * D + e0, x);
        }
        const float* w = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = LPH / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        float y[N];
        if (w) {
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 wv = *reinterpret_cast<const float4*>(w + e0 + i);
                y[i] = x[i] * r * wv.x;
                y[i + 1] = x[i + 1] * r * wv.y;
                y[i + 2] = x[i + 2] * r * wv.z;
                y[i + 3] = x[i + 3] * r * wv.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = x[i];
        }
        float z[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float other = INTERLEAVED ? y[i ^ 1] : __shfl_sync(0xffffffffu, y[i], partner);
            z[i] = rot ? fmaf(y[i], c[i], other * s[i]) : y[i];
        }
        if (!ok) continue;
        if (is_q) {
            V::store(static_cast<T*>(a.q_out) + (row * Hq + h) * D + e0, z);
        } else if (is_k) {
            if (a.k_out) V::store(static_cast<T*>(a.k_out) + (row * Hkv + h) * D + e0, z);
            if (k_page) V::store(k_page + h * a.cache_head_stride + e0, z);
        } else if (v_page) {
            V::store(v_page + h * a.cache_head_stride + e0, x);   // the values go in as they came
        }
    }
}

template <typename T, int D, int RT, bool IL>
cudaError_t launch_rt(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int GPR = kThreads / (D / Vec16<T>::N) / RT;
    const int heads = a.num_heads + (a.slots ? 2 : 1) * a.num_kv_heads;
    const long long row_tiles = (a.rows + RT - 1) / RT;
    // few rows: their heads spread over more blocks, down to one head per lane group, until
    // the grid has about two blocks per SM
    long long shares = 1;
    const long long most = (heads + GPR - 1) / GPR;
    while (shares < most && row_tiles * shares < 296) ++shares;
    norm_rope_kernel<T, D, RT, IL><<<dim3((unsigned)row_tiles, (unsigned)shares), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// One row per block while the rows are few, so that a row's heads spread over all lane
// groups; four rows per block otherwise, which gives each thread one angle.
template <typename T, int D, bool IL>
cudaError_t launch_rows(const NormRopeArgs& a, cudaStream_t stream) {
    return a.rows <= 296 ? launch_rt<T, D, 1, IL>(a, stream) : launch_rt<T, D, 4, IL>(a, stream);
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
