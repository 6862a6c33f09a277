// gdn_attn_tc.cu -- bf16 attention of new tokens over a paged cache on the tensor cores
// (tcgen05 + TMA); the formulas are in gdn_attn.cu, the division of the work in gdn_attn.h.
//
// One persistent CTA per SM walks its stretch of the line of key tiles (128 keys).  Ten
// warps work: a loader, an MMA issuer and two groups of four softmax warps.
//   - A row tile holds 128 / group tokens, each with the query heads of one key head, so
//     shared key heads fill the 128 rows of an MMA with few tokens.
//   - Two streams share the tensor core: while one stream's softmax runs, the other's
//     products do.  A unit of more tokens than a row tile gives each stream a row tile and
//     every key tile serves both; a smaller one (single tokens) has both streams on the
//     same rows, the even and the odd key tiles, merged at its end.
//   - Per stream and key tile: S = Q K^T into 128 TMEM columns; one thread per row reads its
//     128 scores, updates the row's maximum and sum in fp32 and writes P = 2^(S - m) as bf16
//     over them; O += P V with P read from TMEM, V from shared memory as the cache has it.
//   - The maximum that scales P lags: O and the sum are rescaled only when a row's maximum
//     grew by more than 2^8 since (P up to 256 costs bf16 and fp32 nothing), so the pass
//     over O is rare after the first tiles.
//   - Keys outside the context or the window: scores become -infinity by selection, V rows
//     become zero in shared memory, so neither can be anything that matters.  Runs of rows
//     that are wholly outside are not read: TMA fills their boxes with zeros (a page
//     coordinate past the pool).
// P's rounding to bf16 (half a step, 2^-8 at most) matches V's own precision and halves the
// second product's cost against tf32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "gdn_attn.h"
#include "gdn_sm100.h"

namespace gdn {
namespace attn {
namespace {

using namespace sm100;

constexpr int kRows = 128;         // rows of a row tile
constexpr int kKeys = 128;         // keys of a tile
constexpr int kThreads = 384;      // softmax groups: warps 0-3 and 4-7; MMA: 8; loader: 9; walker: 10
// registers per thread: 168 at launch (65536 / 384, in steps of 8), then the softmax warps
// take what the third warpgroup gives back: 2 * 208 + 88 = 3 * 168
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kMaxParts = 148;     // one CTA per SM of a B200
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;      // log2 of the growth of a row's maximum that P absorbs
constexpr int kBlock = kKeys * 128;   // bytes of one 64-column block of a 128-row tile

template <int D>
struct Smem {
    static constexpr int TILE = D * 256;                      // a 128-row tile of D bf16 columns
    static constexpr int STAGES = D == 128 ? 5 : 10;          // K and V tiles in flight, in turn
    static constexpr int Q = 0;
    static constexpr int KV = 2 * TILE;
    static constexpr int EXCH = KV + STAGES * TILE;           // the streams' maxima and sums: float [2][2][128]
    static constexpr int BARS = EXCH + 2048;
    static constexpr int BYTES = BARS + 512;
};

// This CTA's part of a unit, handed by the walker to the other roles.
struct Piece {
    int n;                 // key tiles; 0 = the end
    int b, head;           // sequence and key head
    int row0, toks;        // first row of the unit's tokens in q and o, and their number
    int first_pos;         // position of the first one
    int lo, hi;            // keys that some row sees
    int key0;              // first key of the first tile
    int single;            // one row tile: the streams share it
    int slot;              // where partial results go; -1 = the unit is whole here
    int pad;
};

struct Bars {
    uint64_t q_full, q_free, drain, x_full, x_free;
    uint64_t s_full[2], p_ready[2], o_done[2];
    uint64_t piece_full[2], piece_free[2];
    uint64_t kv_full[10], kv_free[10];
    Piece piece[2];
    uint32_t tmem;
    int abort;             // a wait ran out
    int bad_page;
};
static_assert(sizeof(Bars) <= 512, "the barriers fit their space");

struct Maps {
    CUtensorMap q, k, v;
};

// A whole warp's wait, which ends: false (in every lane) when it ran out or another role
// gave up.
__device__ __forceinline__ bool wait(Bars* b, uint64_t* bar, uint32_t parity) {
    bool done = mbar_try_wait(bar, parity);
    if (!done) {
        const uint64_t t0 = global_timer_ns();
        while (!(done = mbar_try_wait(bar, parity))) {
            if (*reinterpret_cast<volatile int*>(&b->abort)) break;
            if (global_timer_ns() - t0 > kWaitNs) {
                *reinterpret_cast<volatile int*>(&b->abort) = 1;   // reported at the end
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, done);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------- walker
// Walks this CTA's stretch of the line and hands out its pieces, two ahead.
__device__ __forceinline__ void walk_role(const Args& a, Bars* b) {
    const int lane = threadIdx.x & 31;
    const long long per = a.line->per_part;
    long long pos = (long long)blockIdx.x * per;
    const long long end = min(pos + per, a.line->total);
    Unit u = find_unit(a, pos);
    for (unsigned i = 0;; ++i) {
        if (i >= 2 && !wait(b, &b->piece_free[i & 1], (i / 2 - 1) & 1)) return;
        Piece p;
        p.n = 0;
        if (pos < end) {
            const int kt0 = (int)(pos - u.begin), kt1 = (int)min((long long)u.r.tiles, end - u.begin);
            p.n = kt1 - kt0;
            p.b = u.b;
            p.head = u.head;
            p.row0 = u.s.row0 + u.r.tok0;
            p.toks = u.r.toks;
            p.first_pos = u.s.ctx - u.s.qlen + u.r.tok0;
            p.lo = u.r.lo;
            p.hi = u.r.hi;
            p.key0 = (u.r.tile0 + kt0) * kKeys;
            p.single = u.r.toks <= a.block_tokens;
            p.slot = p.n == u.r.tiles ? -1 : (int)part_slot(blockIdx.x, i == 0);
            pos += p.n;
        }
        if (lane == 0) {
            b->piece[i & 1] = p;
            mbar_arrive(&b->piece_full[i & 1]);
        }
        __syncwarp();
        if (p.n == 0) return;
        if (pos < end) next_unit(a, u);
    }
}

// The next piece, for a whole warp of another role; n = 0 at the end or when a role gave up.
struct Pieces {
    unsigned i = 0;
    __device__ __forceinline__ Piece get(Bars* b) {
        Piece p;
        p.n = 0;
        if (wait(b, &b->piece_full[i & 1], (i / 2) & 1)) p = b->piece[i & 1];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&b->piece_free[i & 1]);
        ++i;
        return p;
    }
};

// ------------------------------------------------------------------- loader
template <int D>
__device__ __forceinline__ void load_role(const Args& a, const Maps& maps, uint8_t* smem, Bars* b, int granule) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const int runs = kKeys / granule;           // TMA boxes of one 64-column block
    unsigned ring = 0, units = 0;
    bool ok = true;
    Pieces pieces;
    for (Piece u = pieces.get(b); u.n > 0; u = pieces.get(b)) {
        // Q, once the last piece's scores are done with it
        ok = units == 0 || wait(b, &b->q_free, (units - 1) & 1);
        if (!ok) break;
        const int subs = u.single ? 1 : 2;
        if (lane == 0)
            mbar_arrive_expect_tx(&b->q_full, (uint32_t)(subs * D * 2 * a.group * a.block_tokens));
        __syncwarp();
        if (lane < subs * (D / 64)) {
            const int sub = lane / (D / 64), cb = lane % (D / 64);
            tma_load_3d(smem + S::Q + sub * S::TILE + cb * kBlock, &maps.q, &b->q_full, cb * 64, u.head * a.group,
                        u.row0 + sub * a.block_tokens);
        }
        ++units;
        for (int j = 0; ok && j < u.n; ++j) {
            // this lane's run of rows and its page: past the pool (read as zeros) when the
            // run holds no key of the unit, or the page number is bad
            const int run = lane % runs;
            const int key = u.key0 + j * kKeys + run * granule;
            int page = a.num_pages;
            if (key < u.hi && key + granule > u.lo) {
                const int p = a.page_table[(long long)u.b * a.max_pages + key / a.page_size];
                if (p >= 0 && p < a.num_pages) page = p;
                else *reinterpret_cast<volatile int*>(&b->bad_page) = 1;
            }
            const int in_page = key % a.page_size;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const unsigned st = ring % S::STAGES, ph = ring / S::STAGES;
                ok = ph == 0 || wait(b, &b->kv_free[st], (ph - 1) & 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&b->kv_full[st], S::TILE);
                __syncwarp();
                // a lane per (column block, run); 32 is a multiple of the runs, so a lane's run is its own
                for (int i = lane; i < runs * (D / 64); i += 32) {
                    const int cb = i / runs;
                    tma_load_4d(base + S::KV + st * S::TILE + cb * kBlock + run * granule * 128,
                                kv == 0 ? &maps.k : &maps.v, &b->kv_full[st], cb * 64, u.head, in_page, page);
                }
                __syncwarp();
                ++ring;
            }
        }
    }
    if (!ok) {   // wait for this warp's own copies before the CTA may leave
        const unsigned n = min(ring, (unsigned)S::STAGES);
        for (unsigned i = ring - n; i < ring; ++i) mbar_wait_bounded(&b->kv_full[i % S::STAGES], (i / S::STAGES) & 1, kWaitNs);
        if (units) mbar_wait_bounded(&b->q_full, (units - 1) & 1, kWaitNs);
    }
}

// --------------------------------------------------------------- MMA issuer
template <int D>
__device__ __forceinline__ void mma_role(const Args& a, uint8_t* smem, Bars* b) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem), tm = b->tmem;
    const uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, D, false, true);
    unsigned ring = 0, units = 0, p_count0 = 0, p_count1 = 0;
    bool ok = true;

    auto k_stage = [&](int j) { return (ring + 2 * j) % S::STAGES; };
    auto v_stage = [&](int j) { return (ring + 2 * j + 1) % S::STAGES; };
    auto full = [&](unsigned at) { return wait(b, &b->kv_full[at % S::STAGES], (at / S::STAGES) & 1); };
    // S of stream s = row tile `sub` times the keys in `stage`
    auto scores = [&](int s, int sub, unsigned stage) {
        const uint64_t dq = smem_desc_sw128(base + S::Q + sub * S::TILE, 16, 1024);
        const uint64_t dk = smem_desc_sw128(base + S::KV + stage * S::TILE, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kBlock + (kk & 3) * 32;
            mma_bf16_ss(tm + s * 128, desc_advance(dq, off), desc_advance(dk, off), id_s, kk > 0);
        }
        mma_commit(&b->s_full[s]);
    };
    auto values = [&](int s, unsigned stage, bool first) {
        const uint64_t dv = smem_desc_sw128(base + S::KV + stage * S::TILE, kBlock, 1024);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_bf16_ts(tm + 256 + s * 128, tm + s * 128 + kk * 8, desc_advance(dv, kk * 2048), id_o,
                        !first || kk > 0);
    };

    auto p_ready = [&](int s) {
        const unsigned ph = s ? p_count1++ : p_count0++;
        return wait(b, &b->p_ready[s], ph & 1);
    };

    Pieces pieces;
    for (Piece u = pieces.get(b); u.n > 0; u = pieces.get(b)) {
        const int n = u.n;
        // the V rows of tile j that hold no key of this unit become zero
        auto clear_outside = [&](int j) {
            const int key0 = u.key0 + j * kKeys;
            const int from = max(0, u.lo - key0), to = min(kKeys, u.hi - key0);
            if (from == 0 && to == kKeys) return;
            const uint32_t tile = base + S::KV + v_stage(j) * S::TILE;
            for (int i = lane; i < kKeys * (D / 64); i += 32) {
                const int r = i % kKeys;
                if (r >= from && r < to) continue;
                const uint32_t at = tile + (i / kKeys) * kBlock + r * 128;
#pragma unroll
                for (int c = 0; c < 128; c += 16)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + c), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        ok = wait(b, &b->q_full, units & 1);
        ++units;
        if (!ok) break;
        if (u.single) {
            // stream s: tiles s, s + 2, ...
            for (int j = 0; j < min(n, 2); ++j) {
                ok = ok && full(ring + 2 * j);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    scores(j, 0, k_stage(j));
                    mma_commit(&b->kv_free[k_stage(j)]);
                    if (j + 1 == n) mma_commit(&b->q_free);
                }
                __syncwarp();
            }
            for (int j = 0; ok && j < n; ++j) {
                const int s = j & 1;
                ok = full(ring + 2 * j + 1);
                if (!ok) break;
                clear_outside(j);
                ok = p_ready(s);
                if (ok && j + 2 < n) ok = full(ring + 2 * (j + 2));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    values(s, v_stage(j), j < 2);
                    mma_commit(&b->kv_free[v_stage(j)]);
                    if (j + 2 < n) {
                        scores(s, 0, k_stage(j + 2));
                        mma_commit(&b->kv_free[k_stage(j + 2)]);
                        if (j + 3 == n) mma_commit(&b->q_free);
                    } else {
                        mma_commit(&b->o_done[s]);
                    }
                }
                __syncwarp();
            }
        } else {
            ok = full(ring);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                scores(0, 0, k_stage(0));
                scores(1, 1, k_stage(0));
                mma_commit(&b->kv_free[k_stage(0)]);
                if (n == 1) mma_commit(&b->q_free);
            }
            __syncwarp();
            for (int j = 0; ok && j < n; ++j) {
                const bool next = j + 1 < n;
                ok = full(ring + 2 * j + 1);
                if (ok && next) ok = full(ring + 2 * (j + 1));
                if (!ok) break;
                clear_outside(j);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    ok = ok && p_ready(s);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        values(s, v_stage(j), j == 0);
                        if (s == 1) mma_commit(&b->kv_free[v_stage(j)]);
                        if (next) {
                            scores(s, s, k_stage(j + 1));
                            if (s == 1) {
                                mma_commit(&b->kv_free[k_stage(j + 1)]);
                                if (j + 2 == n) mma_commit(&b->q_free);
                            }
                        } else {
                            mma_commit(&b->o_done[s]);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) break;
        ring += 2 * n;
    }
    // everything issued is complete before the TMEM goes back
    if (elect_one()) {
        mma_commit(&b->drain);
        mbar_wait_bounded(&b->drain, 0, kWaitNs);
    }
    __syncwarp();
}

// ------------------------------------------------------------ softmax groups
template <int D>
__device__ __forceinline__ void softmax_role(const Args& a, uint8_t* smem, Bars* b, int s) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tm = b->tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tm_s = tm + s * 128, tm_o = tm + 256 + s * 128;
    float* exch = reinterpret_cast<float*>(smem + S::EXCH);
    const float sl = a.scale * 1.4426950408889634f;
    unsigned s_count = 0, o_count = 0, x_count = 0;
    bool ok = true;
    Pieces pieces;
    for (Piece u = pieces.get(b); u.n > 0; u = pieces.get(b)) {
        const int sub = u.single ? 0 : s;
        const int toks = min(a.block_tokens, u.toks - sub * a.block_tokens);
        const int rows = toks * a.group;
        const int first_pos = u.first_pos + sub * a.block_tokens;
        const int top_key = row < rows ? first_pos + row / a.group : -1;     // keys [low_key, top_key] are seen
        const int low_key = a.window > 0 ? max(0, top_key - a.window + 1) : 0;
        // keys that every row of the tile sees: [all_lo, all_hi]
        const int all_hi = first_pos;
        const int all_lo = a.window > 0 ? max(0, first_pos + toks - a.window) : 0;
        const bool active = quarter * 32 < rows;   // this warp has rows
        float m = -INFINITY, l = 0.0f;
        bool any_tile = false;
        for (int j = u.single ? s : 0; j < u.n; j += u.single ? 2 : 1) {
            ok = wait(b, &b->s_full[s], s_count++ & 1);
            if (!ok) break;
            tc_fence_after();
            if (active) {
                const int key0 = u.key0 + j * kKeys;
                float x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tm_s + c * 32, x + c * 32);
                tmem_wait_ld();
                if (key0 < all_lo || key0 + kKeys - 1 > all_hi) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        x[i] = key0 + i >= low_key && key0 + i <= top_key ? x[i] : -INFINITY;
                }
                float t0 = x[0], t1 = x[1], t2 = x[2], t3 = x[3];
#pragma unroll
                for (int i = 4; i < 128; i += 4) {
                    t0 = fmaxf(t0, x[i]);
                    t1 = fmaxf(t1, x[i + 1]);
                    t2 = fmaxf(t2, x[i + 2]);
                    t3 = fmaxf(t3, x[i + 3]);
                }
                const float top = fmaxf(m, fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)));
                if (__any_sync(0xffffffffu, (top - m) * sl > kLazy)) {
                    const float f = m == -INFINITY ? 0.0f : ex2((m - top) * sl);
                    l *= f;
                    m = top;
                    if (any_tile) {   // the last product into O is complete: this tile's scores came behind it
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tm_o + c * 16, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(tm_o + c * 16, o);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.0f : -m * sl;
                float l0 = 0.0f, l1 = 0.0f, l2 = 0.0f, l3 = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float e0 = ex2(fmaf(x[32 * c + 2 * i], sl, off)), e1 = ex2(fmaf(x[32 * c + 2 * i + 1], sl, off));
                        const float e2 = ex2(fmaf(x[32 * c + 2 * i + 2], sl, off)), e3 = ex2(fmaf(x[32 * c + 2 * i + 3], sl, off));
                        l0 += e0;
                        l1 += e1;
                        l2 += e2;
                        l3 += e3;
                        p[i] = pack(e0, e1);
                        p[i + 1] = pack(e2, e3);
                    }
                    tmem_st16(tm_s + c * 16, p);
                }
                l += (l0 + l1) + (l2 + l3);
                tmem_wait_st();
            }
            any_tile = true;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->p_ready[s]);
        }
        if (ok && any_tile) ok = wait(b, &b->o_done[s], o_count++ & 1);
        if (!ok) break;
        if (u.single) {   // both streams' outputs are complete, their maxima and sums exchanged
            exch[s * 256 + row] = any_tile && active ? m : -INFINITY;
            exch[s * 256 + 128 + row] = any_tile && active ? l : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->x_full);
            ok = wait(b, &b->x_full, x_count & 1);
            if (!ok) break;
        }
        tc_fence_after();
        const int h = row % a.group;
        const long long orow =
            (long long)(u.row0 + sub * a.block_tokens + row / a.group) * a.num_heads + u.head * a.group + h;
        const long long prow = (long long)u.slot * (2 * kRows) + sub * kRows + row;
        const bool whole = u.slot < 0;
        if (active) {
            // weights of the two streams' sums (the other stream has other rows: 0)
            float f0 = 1.0f, f1 = 0.0f, sum = l, top = m;
            bool both = false;
            if (u.single) {
                const float m0 = exch[row], l0 = exch[128 + row], m1 = exch[256 + row], l1 = exch[256 + 128 + row];
                top = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.0f : ex2((m0 - top) * sl);
                f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - top) * sl);
                sum = l0 * f0 + l1 * f1;
                both = u.n > 1;          // the second stream had a tile
            }
            const float inv = sum > 0.0f || isnan(sum) ? 1.0f / sum : 0.0f;
            f0 *= inv;
            f1 *= inv;
            // single: this group takes half of the columns, of both streams
            const int c0 = u.single ? s * (D / 64) : 0, c1 = u.single ? c0 + D / 64 : D / 32;
            const uint32_t from = u.single ? tm + 256 : tm_o;
            for (int c = c0; c < c1; ++c) {
                float o[32];
                tmem_ld32(from + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f0;
                if (both) {
                    float z[32];
                    tmem_ld32(from + 128 + c * 32, z);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(z[i], f1, o[i]);
                }
                if (row < rows) {
                    if (whole) {
                        uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + orow * D + c * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            to[i] = make_uint4(pack(o[8 * i], o[8 * i + 1]), pack(o[8 * i + 2], o[8 * i + 3]),
                                               pack(o[8 * i + 4], o[8 * i + 5]), pack(o[8 * i + 6], o[8 * i + 7]));
                    } else {
                        float4* to = reinterpret_cast<float4*>(a.part_o + prow * D + c * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
            if (row < rows && (!u.single || s == 0)) {
                const float lse2 = sum > 0.0f || isnan(sum) ? top * sl + log2f(sum) : -INFINITY;
                if (!whole) a.part_lse[prow] = lse2;
                else if (a.lse) a.lse[orow] = lse2 * kLn2;
            }
        }
        // both groups have read both streams' sums and outputs before either stream goes on
        tc_fence_before();
        if (u.single) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->x_free);
            ok = wait(b, &b->x_free, x_count++ & 1);
            if (!ok) break;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const Args a, const __grid_constant__ Maps maps, int granule) {
    using S = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars* b = reinterpret_cast<Bars*>(smem + S::BARS);
    const int warp = threadIdx.x >> 5;
    if ((int)blockIdx.x >= a.line->parts) return;
    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the runtime places the block's memory so
        if (threadIdx.x == 0) tag_merge_inline(&a.ws->status, a.epoch, kStatusBounds, false);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(&b->q_full, 1);
        mbar_init(&b->q_free, 1);
        mbar_init(&b->drain, 1);
        mbar_init(&b->x_full, 8);
        mbar_init(&b->x_free, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&b->s_full[s], 1);
            mbar_init(&b->p_ready[s], 4);
            mbar_init(&b->o_done[s], 1);
            mbar_init(&b->piece_full[s], 1);
            mbar_init(&b->piece_free[s], 10);   // the softmax, MMA and loader warps
        }
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&b->kv_full[i], 1);
            mbar_init(&b->kv_free[i], 1);
        }
        b->abort = b->bad_page = 0;
        mbar_fence_init();
    }
    if (warp == 8) {
        tmem_alloc(&b->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 9 && elect_one()) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax_role<D>(a, smem, b, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) mma_role<D>(a, smem, b);
        else if (warp == 9) load_role<D>(a, maps, smem, b, granule);
        else if (warp == 10) walk_role(a, b);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(b->tmem, 512);
        const unsigned int bits = (b->abort ? kStatusTimeout : 0u) | (b->bad_page ? kStatusMismatch : 0u);
        if (bits && elect_one()) tag_merge_inline(&a.ws->status, a.epoch, bits, false);
    }
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const cuuint32_t es[4] = {1, 1, 1, 1};
    const EncodeTiledFn enc = tensor_map_encoder();
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_typed(const Args& a, const Maps& maps, int granule, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e =
        ensure_smem_limit(reinterpret_cast<const void*>(attn_tc_kernel<D>), Smem<D>::BYTES, smem_set);
    if (e != cudaSuccess) return e;
    attn_tc_kernel<D><<<kMaxParts, kThreads, Smem<D>::BYTES, stream>>>(a, maps, granule);
    return cudaGetLastError();
}

}  // namespace

Shape shape_tc() { return Shape{kRows, 2, kKeys, kMaxParts, 2}; }

cudaError_t launch_tc(const Args& a, cudaStream_t stream) {
    // rows of one page that a tile's box can hold: the largest power of two that divides the
    // page, so that no box crosses a page or a tile
    int granule = kKeys;
    while (a.page_size % granule != 0) granule /= 2;
    Maps maps;
    const cuuint64_t D = (cuuint64_t)a.dim;
    {
        const cuuint64_t dims[3] = {D, (cuuint64_t)a.num_heads, (cuuint64_t)a.rows};
        const cuuint64_t strides[2] = {D * 2, (cuuint64_t)a.rs_q * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.block_tokens};
        if (!encode(&maps.q, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const cuuint64_t dims[4] = {D, (cuuint64_t)a.num_kv_heads, (cuuint64_t)a.page_size, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.head_stride * 2, (cuuint64_t)a.row_stride * 2,
                                   (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)granule, 1};
    if (!encode(&maps.k, a.k, 4, dims, strides, box) || !encode(&maps.v, a.v, 4, dims, strides, box))
        return cudaErrorInvalidValue;
    return a.dim == 64 ? launch_typed<64>(a, maps, granule, stream) : launch_typed<128>(a, maps, granule, stream);
}

}  // namespace attn
}  // namespace gdn
