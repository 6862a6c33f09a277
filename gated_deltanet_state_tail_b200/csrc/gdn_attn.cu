// gdn_attn.cu -- attention of a chunk of new tokens over a paged cache: the layout of
// the work for many sequences (gdn_attn.h), and the fp32 attention kernel.
//
// Per new token i of a sequence with n new tokens and context L (position p = L - n + i)
// and query head h, over the keys j in (p - window, p], j >= 0, of key head h / group:
//   o = sum_j softmax_j(scale q . k_j) v_j,    lse = log sum_j exp(scale q . k_j)
// in one pass over the keys with a running maximum and sum.  A row without keys gives
// o = 0 and lse = -infinity; one whose scores are all -infinity o = NaN and the same lse.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "gdn_attn.h"
#include "gdn_f32x2.h"

namespace gdn {
namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ the line
// One block.  A warp per sequence adds up its units' lengths; a scan over the
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
    for (int b = warp; b < a.batch; b += 32) {
        bool good;
        const Seq s = load_seq<true>(a, b, good);
        if (lane == 0) {
            a.seqs[b] = s;
            if (!good) report(a, kStatusMismatch);
        }
    }
    __syncthreads();
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        const long long n = b < a.batch ? a.seqs[b].head_len * a.num_kv_heads : 0;
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
    if (threadIdx.x == 0) *a.line = make_line(a, carry);
}

// ------------------------------------------------------------- fp32 attention
// 64 rows x 64 keys per tile on the CUDA cores.  128 threads: thread (ty, tx) holds the
// scores of rows 8 ty .. 8 ty + 7 and keys tx + 16 j, and the outputs of those rows and
// columns 4 tx + 64 j, so that 12 reads of shared memory feed 128 multiply-adds (with 4 x 4
// scores a thread and 256 threads, 8 fed 64).  K of the next tile is copied (cp.async)
// while P V runs, V while the scores do; 113 KB for d = 128, so that two CTAs share an SM.
// The rows' places in the pages are worked out once per tile, a thread per row, and kept in
// the padding of K's rows.  Bound by the fp32 pipe (4 d flops per row and key).
//
// Units of at most 8 rows (single tokens) would leave most of those tiles empty; they have
// all threads on the keys: two lanes per key for the scores, a warp per two rows for the
// softmax, and for P V a thread per column and share of the keys.  Bound by HBM then.
constexpr int kRows = 64, kKeys = 64, kThreads = 128, kFew = 8;
constexpr int kWarps = kThreads / 32, kTR = kRows / (kThreads / 16);   // kTR: rows of a thread
template <int D>
struct SimtSmem {
    // columns of q and p exchange their neighbouring fours (c ^ 4) in every other eight rows:
    // a warp reads two rows eight apart at once, which would share their banks
    float q[kRows][D];
    // padded: float4 reads of 8 rows hit 32 banks; the padding holds two places in the
    // pages, of this tile's row and of the next one's
    float k[kKeys][D + 4];
    float v[kKeys][D];
    float p[kRows][kKeys];                         // few rows: [8][64] and behind them
    __device__ float* keep() { return p[kFew]; }   // 2^(old maximum - new) of each row
    __device__ float* inv() { return p[kFew + 1]; }
    __device__ long long& place(int r, int slot) { return *reinterpret_cast<long long*>(&k[r][D + 2 * slot]); }
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Row r of a split unit merged by a warp, its columns over the lanes, eight parts read at
// once; every part has the weight 2^(its log-sum).
template <int D>
__device__ __forceinline__ void merge_row(const Args& a, const Split& sp, int r, bool sees, float* to, float* lse) {
    constexpr int AHEAD = 8;
    const int lane = threadIdx.x & 31, col = 4 * lane;
    float top = -INFINITY, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = sp.first; p0 <= sp.last; p0 += AHEAD) {
        float w[AHEAD];
        float4 x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const long long row = (p0 + i <= sp.last ? sp.slot(p0 + i) : 0) * kRows + r;
            w[i] = p0 + i <= sp.last ? __ldcg(a.part_lse + row) : -INFINITY;
            x[i] = p0 + i <= sp.last && col < D ? __ldcg(reinterpret_cast<const float4*>(a.part_o + row * D + col))
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        float t = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) t = fmaxf(t, w[i]);
        const float ref = t == -INFINITY ? 0.0f : t, keep = exp2f(top - ref);
        top = t;
        sum *= keep;
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float f = exp2f(w[i] - ref);
            sum += f;
            acc.x = fmaf(f, x[i].x, acc.x);
            acc.y = fmaf(f, x[i].y, acc.y);
            acc.z = fmaf(f, x[i].z, acc.z);
            acc.w = fmaf(f, x[i].w, acc.w);
        }
    }
    const float inv = inverse_sum(sum, sees);   // a NaN part makes the row NaN
    if (col < D)
        *reinterpret_cast<float4*>(to + col) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (lse && lane == 0) *lse = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) simt_kernel(const Args a) {
    extern __shared__ __align__(16) float smem_raw[];
    SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem_raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (a.merge_kernel && tid == 0) a.splits[blockIdx.x].last = -1;
    const Line ln = get_line<kThreads>(a, reinterpret_cast<long long*>(smem_raw));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((int)blockIdx.x >= ln.parts) return;
    const long long per = ln.per_part;
    const long long start = (long long)blockIdx.x * per, end = min(start + per, ln.total);
    const StoredSeqs seqs{a};
    Unit u = find_unit(a, seqs, start);
    const float scale = a.scale * kLog2e;
    for (;; next_unit(a, seqs, u)) {
        if (start - u.begin >= u.r.tiles) {   // only the unit's extra is in this stretch
            if (unit_end(a, u) >= end) break;
            continue;
        }
        const bool begins = u.begin <= start;
        const int kt0 = (int)max(0ll, start - u.begin);
        const int kt1 = (int)min((long long)u.r.tiles, end - u.begin);
        const int rows = u.r.toks * a.group;
        const int first_pos = u.s.ctx - u.s.qlen + u.r.tok0;
        // where the rows of the tile at key0 are in the pools; -1 outside the unit's keys and
        // for a bad page number, both of which read as zeros
        auto find_places = [&](int key0, int slot) {
            if (tid >= kKeys) return;
            const int key = key0 + tid;
            long long at = -1;
            if (key >= u.r.lo && key < u.r.hi) {
                const int page = a.page_table[(long long)u.b * a.max_pages + key / a.page_size];
                if (page >= 0 && page < a.num_pages)
                    at = (long long)page * a.page_stride + (long long)(key % a.page_size) * a.row_stride +
                         (long long)u.head * a.head_stride;
                else
                    report(a, kStatusMismatch);
            }
            sm.place(tid, slot) = at;
        };
        auto copy_rows = [&](const void* base, float* dst, int ld, int slot) {
#pragma unroll 8
            for (int n = 0; n < kKeys * (D / 4) / kThreads; ++n) {
                const int i = tid + n * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
                const long long at = sm.place(r, slot);
                copy16(dst + r * ld + c, static_cast<const float*>(base) + (at >= 0 ? at + c : 0), at >= 0);
            }
        };
        __syncthreads();   // the last unit's reads of shared memory are over
        find_places((u.r.tile0 + kt0) * kKeys, 0);
        // queries and the first tile's keys
#pragma unroll
        for (int n = 0; n < kRows * (D / 4) / kThreads; ++n) {
            const int i = tid + n * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
            const bool on = r < rows;
            copy16(&sm.q[r][c ^ (4 * ((r / kTR) & 1))],
                   static_cast<const float*>(a.q) +
                       (on ? (long long)(u.s.row0 + u.r.tok0 + r / a.group) * a.rs_q +
                                 (long long)(u.head * a.group + r % a.group) * D + c
                           : 0),
                   on);
        }
        __syncthreads();   // the places are in
        copy_rows(a.k, &sm.k[0][0], D + 4, 0);
        copies_commit();
        // Tiles with keys that some row does not see: P is 0 there, but 0 times an infinity or a
        // NaN is not.  If such a tile of V holds one, each row skips the keys that it does not
        // see (a thread looks through its share of the tile; the block agrees).
        const int all_lo = first_key(a, first_pos + u.r.toks - 1);
        auto careful = [&](int key0) {
            if (u.r.toks == 1 || (key0 + kKeys - 1 <= first_pos && key0 >= all_lo)) return false;   // uniform
            float acc = 0.0f;
#pragma unroll 4
            for (int i = tid; i < kKeys * D / 4; i += kThreads) {
                const float4 x = reinterpret_cast<const float4*>(&sm.v[0][0])[i];
                acc = fmaf(x.x, 0.0f, fmaf(x.y, 0.0f, fmaf(x.z, 0.0f, fmaf(x.w, 0.0f, acc))));
            }
            return __syncthreads_or(acc != 0.0f) != 0;   // zero or NaN
        };
        const bool whole = kt0 == 0 && kt1 == u.r.tiles;
        auto out_row = [&](int r) {
            return (long long)(u.s.row0 + u.r.tok0 + r / a.group) * a.num_heads + u.head * a.group + r % a.group;
        };
        if (rows <= kFew) {
            const int lane = tid & 31, warp = tid >> 5;     // warp w has rows w and w + kWarps
            constexpr int PARTS = kThreads / kKeys;         // lanes of a key, for the scores
            constexpr int SHARES = kThreads / D;            // of the keys, for P V
            const int col = tid % D, share = tid / D;
            float m[kFew / kWarps], l[kFew / kWarps], acc[kFew];
#pragma unroll
            for (int j = 0; j < kFew / kWarps; ++j) m[j] = -INFINITY, l[j] = 0.0f;
#pragma unroll
            for (int r = 0; r < kFew; ++r) acc[r] = 0.0f;
            for (int kt = kt0; kt < kt1; ++kt) {
                const int key0 = (u.r.tile0 + kt) * kKeys, slot = (kt - kt0) & 1;
                copy_rows(a.v, &sm.v[0][0], D, slot);
                copies_commit();
                if (kt + 1 < kt1) find_places(key0 + kKeys, slot ^ 1);
                copies_wait<1>();
                __syncthreads();                            // K (and Q) are in
                {
                    const int key = tid / PARTS, part = tid % PARTS;
                    float sc[kFew];
#pragma unroll
                    for (int r = 0; r < kFew; ++r) sc[r] = 0.0f;
#pragma unroll 4
                    for (int c = 4 * part; c < D; c += 4 * PARTS) {
                        const float4 kv = *reinterpret_cast<const float4*>(&sm.k[key][c]);
#pragma unroll
                        for (int r = 0; r < kFew; ++r)
                            if (r < rows) {
                                const float4 qv = *reinterpret_cast<const float4*>(&sm.q[r][c]);
                                sc[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, sc[r]))));
                            }
                    }
#pragma unroll
                    for (int r = 0; r < kFew; ++r) {
#pragma unroll
                        for (int d = PARTS / 2; d > 0; d >>= 1) sc[r] += __shfl_xor_sync(0xffffffffu, sc[r], d);
                        if (r % PARTS == part) sm.p[r][key] = sc[r] * scale;
                    }
                }
                __syncthreads();                            // the scores are in, K is read
                if (kt + 1 < kt1) copy_rows(a.k, &sm.k[0][0], D + 4, slot ^ 1);
                copies_commit();
#pragma unroll
                for (int j = 0; j < kFew / kWarps; ++j) {
                    const int r = warp + j * kWarps;
                    if (r >= rows) break;
                    const int top_key = first_pos + r / a.group;
                    const int low_key = first_key(a, top_key);
                    float s0 = sm.p[r][lane], s1 = sm.p[r][lane + 32];
                    const int k0 = key0 + lane, k1 = k0 + 32;
                    s0 = k0 >= low_key && k0 <= top_key ? s0 : -INFINITY;
                    s1 = k1 >= low_key && k1 <= top_key ? s1 : -INFINITY;
                    float top = fmaxf(m[j], fmaxf(s0, s1));
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    const float keep = exp2f(m[j] - ref), p0 = exp2f(s0 - ref), p1 = exp2f(s1 - ref);
                    m[j] = top;
                    l[j] = l[j] * keep + (p0 + p1);               // this lane's share of the row's sum
                    sm.p[r][lane] = p0;
                    sm.p[r][lane + 32] = p1;
                    if (lane == 0) sm.keep()[r] = keep;
                }
                copies_wait<1>();
                __syncthreads();                            // V and P are in
                const bool skip = careful(key0);
#pragma unroll
                for (int r = 0; r < kFew; ++r)
                    if (r < rows) acc[r] *= sm.keep()[r];
                if (skip) {
#pragma unroll 1
                    for (int n = 0; n < kKeys / SHARES; ++n) {
                        const int k = share * (kKeys / SHARES) + (n ^ 3);   // in the order of the sums below
                        const float x = sm.v[k][col];
#pragma unroll
                        for (int r = 0; r < kFew; ++r) {
                            const int top_key = first_pos + r / a.group;
                            if (r < rows && key0 + k <= top_key && (a.window == 0 || key0 + k > top_key - a.window))
                                acc[r] = fmaf(sm.p[r][k], x, acc[r]);
                        }
                    }
                } else
#pragma unroll 2
                for (int key = share * (kKeys / SHARES); key < (share + 1) * (kKeys / SHARES); key += 4) {
                    const float v0 = sm.v[key][col], v1 = sm.v[key + 1][col], v2 = sm.v[key + 2][col],
                                v3 = sm.v[key + 3][col];
#pragma unroll
                    for (int r = 0; r < kFew; ++r)
                        if (r < rows) {
                            const float4 pv = *reinterpret_cast<const float4*>(&sm.p[r][key]);
                            acc[r] = fmaf(pv.x, v0, fmaf(pv.y, v1, fmaf(pv.z, v2, fmaf(pv.w, v3, acc[r]))));
                        }
                }
                __syncthreads();                            // V and P are read
            }
            // the shares of the keys join in the K buffer
            float* part = &sm.k[0][0];
#pragma unroll
            for (int r = 0; r < kFew; ++r) part[(share * kFew + r) * D + col] = acc[r];
#pragma unroll
            for (int j = 0; j < kFew / kWarps; ++j) {
                const int r = warp + j * kWarps;
                if (r >= rows) break;
                float sum = l[j];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == 0) {
                    const float lse2 = sum == 0.0f ? -INFINITY : m[j] + log2f(sum);
                    sm.inv()[r] = inverse_sum(sum, whole && first_pos + r / a.group >= 0);
                    if (!whole) a.part_lse[part_slot(blockIdx.x, begins) * kRows + r] = lse2;
                    else if (a.lse) a.lse[out_row(r)] = lse2 * kLn2;
                }
            }
            __syncthreads();
            for (int i = tid; i < rows * D; i += kThreads) {
                const int r = i / D, c = i % D;
                float x = 0.0f;
#pragma unroll
                for (int n = 0; n < SHARES; ++n) x += part[(n * kFew + r) * D + c];
                (whole ? static_cast<float*>(a.o) + out_row(r) * D
                       : a.part_o + (part_slot(blockIdx.x, begins) * kRows + r) * D)[c] = x * sm.inv()[r];
            }
        } else {
            float m[kTR], l[kTR];
            Pair o[kTR][D / 32];                       // columns 4 tx + 64 j and the next, and the two behind them
            int top_key[kTR], low_key[kTR];                // keys [low, top] are seen
#pragma unroll
            for (int i = 0; i < kTR; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.0f;
                top_key[i] = first_pos + (kTR * ty + i) / a.group;
                low_key[i] = first_key(a, top_key[i]);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) o[i][j] = 0ull;
            }
            const int swap = 4 * (ty & 1);
            const bool active = (kTR * (ty & ~1)) < rows;   // warp-uniform: some row of this warp is a real one
            for (int kt = kt0; kt < kt1; ++kt) {
                const int key0 = (u.r.tile0 + kt) * kKeys, slot = (kt - kt0) & 1;
                copy_rows(a.v, &sm.v[0][0], D, slot);     // its last readers passed the barrier below
                copies_commit();
                if (kt + 1 < kt1) find_places(key0 + kKeys, slot ^ 1);
                copies_wait<1>();
                __syncthreads();                          // K (and Q) are in
                float s[kTR][4];
                if (active) {
                    Pair sum[kTR][4];   // of the even and the odd columns
#pragma unroll
                    for (int i = 0; i < kTR; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum[i][j] = 0ull;
#pragma unroll 2
                    for (int c = 0; c < D; c += 4) {
                        ulonglong2 qv[kTR], kv[4];
#pragma unroll
                        for (int i = 0; i < kTR; ++i) qv[i] = *reinterpret_cast<const ulonglong2*>(&sm.q[kTR * ty + i][c ^ swap]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
                        for (int i = 0; i < kTR; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                sum[i][j] = fma2(qv[i].y, kv[j].y, fma2(qv[i].x, kv[j].x, sum[i][j]));
                    }
#pragma unroll
                    for (int i = 0; i < kTR; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 t = unpair(sum[i][j]);
                            s[i][j] = t.x + t.y;
                        }
#pragma unroll
                    for (int i = 0; i < kTR; ++i) {
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
                            sm.p[kTR * ty + i][(tx + 16 * j) ^ swap] = s[i][j];
                        }
                        l[i] = l[i] * keep + sum;         // this lane's share of the row's sum
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) o[i][j] = mul2(o[i][j], pair(keep, keep));
                    }
                }
                __syncthreads();                          // K is read
                if (kt + 1 < kt1) copy_rows(a.k, &sm.k[0][0], D + 4, slot ^ 1);
                copies_commit();
                copies_wait<1>();
                __syncthreads();                          // V is in, P is written
                const bool skip = careful(key0);
                if (active && skip) {
#pragma unroll 1
                    for (int c = 0; c < kKeys; ++c) {
                        ulonglong2 x[D / 64];
#pragma unroll
                        for (int j = 0; j < D / 64; ++j)
                            x[j] = *reinterpret_cast<const ulonglong2*>(&sm.v[c][4 * tx + 64 * j]);
#pragma unroll
                        for (int i = 0; i < kTR; ++i) {
                            if (key0 + c > top_key[i] || key0 + c < low_key[i]) continue;
                            const float p = sm.p[kTR * ty + i][c ^ swap];
#pragma unroll
                            for (int j = 0; j < D / 64; ++j) {
                                o[i][2 * j] = fma2(pair(p, p), x[j].x, o[i][2 * j]);
                                o[i][2 * j + 1] = fma2(pair(p, p), x[j].y, o[i][2 * j + 1]);
                            }
                        }
                    }
                } else if (active) {
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 4) {
                        float4 pv[kTR];
#pragma unroll
                        for (int i = 0; i < kTR; ++i) pv[i] = *reinterpret_cast<const float4*>(&sm.p[kTR * ty + i][c ^ swap]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            ulonglong2 x[D / 64];
#pragma unroll
                            for (int j = 0; j < D / 64; ++j)
                                x[j] = *reinterpret_cast<const ulonglong2*>(&sm.v[c + e][4 * tx + 64 * j]);
#pragma unroll
                            for (int i = 0; i < kTR; ++i) {
                                const float p = e == 0 ? pv[i].x : e == 1 ? pv[i].y : e == 2 ? pv[i].z : pv[i].w;
                                const Pair pp = pair(p, p);
#pragma unroll
                                for (int j = 0; j < D / 64; ++j) {
                                    o[i][2 * j] = fma2(pp, x[j].x, o[i][2 * j]);
                                    o[i][2 * j + 1] = fma2(pp, x[j].y, o[i][2 * j + 1]);
                                }
                            }
                        }
                    }
                }
                __syncthreads();                          // V and P are read
            }
            if (active) {
#pragma unroll
                for (int i = 0; i < kTR; ++i) {
                    float sum = l[i];
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    const float inv = inverse_sum(sum, whole && top_key[i] >= 0);
                    const float lse2 = sum == 0.0f ? -INFINITY : m[i] + log2f(sum);
                    const int r = kTR * ty + i;
                    if (r >= rows) continue;
                    const long long orow = out_row(r), prow = part_slot(blockIdx.x, begins) * kRows + r;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const float2 lo = unpair(o[i][2 * j]), hi = unpair(o[i][2 * j + 1]);
                        *reinterpret_cast<float4*>((whole ? static_cast<float*>(a.o) + orow * D : a.part_o + prow * D) +
                                                   4 * tx + 64 * j) =
                            make_float4(lo.x * inv, lo.y * inv, hi.x * inv, hi.y * inv);
                    }
                    if (tx == 0) {
                        if (!whole) a.part_lse[prow] = lse2;
                        else if (a.lse) a.lse[orow] = lse2 * kLn2;
                    }
                }
            }
        }
        if (!whole) {
            const Split sp = split_of(u, per);
            if (rows <= kFew) {
                // the block that brings the unit's last part merges it; the part counts as in once
                // every thread has written its share
                __threadfence();
                __syncthreads();
                if (__syncthreads_or(tid == 0 && claim_arrivals(a, sp, 0) && arrive_last(a, sp, 0)))
                    for (int r = tid >> 5; r < rows; r += kWarps)
                        merge_row<D>(a, sp, r, first_pos + r / a.group >= 0, static_cast<float*>(a.o) + out_row(r) * D,
                                     a.lse ? a.lse + out_row(r) : nullptr);
            } else if (sp.first == (int)blockIdx.x && sp.last > sp.first) {
                if (tid == 0)
                    a.splits[blockIdx.x] = SplitUnit{sp.last, sp.from_start, u.s.row0 + u.r.tok0, u.r.toks, u.head, first_pos, {}};
            }
        }
        if (unit_end(a, u) >= end) break;
    }
}

// The units of many rows that the cuts split: block (i, y) the one that CTA i of the
// attention kernel began, a warp per row.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const SplitUnit u = a.splits[blockIdx.x];
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (!to_merge(u, blockIdx.x, a.shape.max_parts, a.block_tokens, a.rows, a.num_kv_heads) || r >= u.toks * a.group) return;
    const long long row = (long long)(u.row0 + r / a.group) * a.num_heads + u.head * a.group + r % a.group;
    merge_row<D>(a, Split{(int)blockIdx.x, u.last, u.from_start != 0}, r, u.first_pos + r / a.group >= 0,
                 static_cast<float*>(a.o) + row * D, a.lse ? a.lse + row : nullptr);
}

template <int D>
cudaError_t launch_simt_typed(const Args& a, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e =
        ensure_smem_limit(reinterpret_cast<const void*>(simt_kernel<D>), (int)sizeof(SimtSmem<D>), smem_set);
    if (e != cudaSuccess) return e;
    simt_kernel<D><<<a.shape.max_parts, kThreads, sizeof(SimtSmem<D>), stream>>>(a);
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess || !a.merge_kernel) return launched;
    return launch_merge(merge_kernel<D>, dim3((unsigned)a.shape.max_parts - 1, kRows / 8), a, stream);
}

}  // namespace

// two CTAs per SM of a B200; unit_extra: a prompt of 2048 tokens took 275, 266 and 268 us with
// 0, 1 and 2
constexpr Shape kSimtShape{kRows, 1, kKeys, 296, kThreads, 1, 1, kFew};

cudaError_t launch_simt(const Args& a, cudaStream_t stream) {
    return a.dim == 64 ? launch_simt_typed<64>(a, stream) : launch_simt_typed<128>(a, stream);
}

}  // namespace attn

attn::Shape paged_attention_shape(int dtype, int) { return dtype == GDN_F32 ? attn::kSimtShape : attn::shape_tc(); }

attn::Layout paged_attention_layout(int dtype, int dim, int batch) {
    constexpr size_t kMostParts = 296;   // of either kernel
    const attn::Shape sh = paged_attention_shape(dtype, dim);
    const size_t rows = (size_t)2 * sh.max_parts * sh.subs * sh.sub_rows;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    // What lasts from call to call (the arrival counts, back at zero after each) has its place
    // whatever the sizes; the sequences, whose number varies, come last.
    attn::Layout l;
    l.line = sizeof(WorkspaceHeader);
    l.arrivals = l.line + sizeof(attn::Line);
    l.splits = l.arrivals + up(sizeof(unsigned long long) * kMostParts * attn::kArrivals);
    l.part_lse = l.splits + up(sizeof(attn::SplitUnit) * kMostParts);
    l.part_o = l.part_lse + up(sizeof(float) * rows);
    l.seqs = l.part_o + up(sizeof(float) * rows * dim);
    l.bytes = l.seqs + up(sizeof(attn::Seq) * (size_t)batch);
    return l;
}

cudaError_t launch_paged_attention(const attn::Args& args, cudaStream_t stream) {
    attn::Args a = args;
    // Every CTA lays out the line itself when a thread per sequence suffices and none has
    // many token blocks to go through (32: under a microsecond); a launch less.
    const long long step = (long long)a.block_tokens * a.shape.subs;
    a.line_inline = a.batch <= a.shape.threads && (a.rows + step - 1) / step <= 32;
    if (a.line_inline && a.batch <= 32 && a.dtype == GDN_BF16) a.line_inline = 2;   // no block barrier before the first loads
    // two row tiles in a unit, or more rows than its last part's CTA merges
    a.merge_kernel = a.shape.subs > 1 ? a.rows > a.block_tokens
                                      : std::min(a.rows, step) * a.group > a.shape.few_rows;
    if (!a.line_inline) {
        attn::line_kernel<<<1, 1024, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return a.dtype == GDN_F32 ? attn::launch_simt(a, stream) : attn::launch_tc(a, stream);
}

}  // namespace gdn
