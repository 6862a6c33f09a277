// gdn_attn_tc.cu -- bf16 attention of new tokens over a paged cache on the tensor cores
// (tcgen05 + TMA); the formulas are in gdn_attn.cu, the division of the work in gdn_attn.h.
//
// One persistent CTA per SM walks its stretch of the line of key tiles (128 keys).  Twelve
// warps work: a loader, two MMA issuers, a walker along the line and two groups of four
// softmax warps.
//   - A row tile holds 128 / group tokens, each with the query heads of one key head, so
//     shared key heads fill the 128 rows of an MMA with few tokens.
//   - Two streams share the tensor core: while one stream's softmax runs, the other's
//     products do.  A unit of more tokens than a row tile gives each stream a row tile, and
//     its steps are the halves (64 keys) of each key tile; a smaller one (single tokens) has
//     both streams on the same rows, a half of each key tile each, merged at its end.
//   - Per stream and step: S = Q K^T into 64 TMEM columns, one of two buffers, so that the
//     next step's scores are there when a softmax ends; one thread per row reads its 64
//     scores, updates the row's maximum and sum in fp32 and writes P = 2^(S - m) as bf16 over
//     them; O += P V with P read from TMEM, V from shared memory as the cache has it.  An MMA
//     of 64 columns with both operands in shared memory takes 48 clocks instead of 32 (a
//     probe: shared memory feeds it 128 bytes a clock), so a pair of row tiles costs 2480
//     tensor core clocks per 128 keys instead of 2048; but steps of 128 keys leave no TMEM for
//     a second buffer, and the chain softmax -> products -> softmax took 3460.
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
#include "gdn_f32x2.h"
#include "gdn_sm100.h"

namespace gdn {
namespace attn {
namespace {

using namespace sm100;

constexpr int kRows = 128;         // rows of a row tile
constexpr int kKeys = 128;         // keys of a tile
constexpr int kStep = 64;          // keys of a softmax step
constexpr int kThreads = 384;      // softmax groups: warps 0-3 and 4-7; MMA: 8 and 9; loader: 10; walker: 11
constexpr int kMaxParts = 148;     // one CTA per SM of a B200
constexpr uint64_t kWaitNs = 1000000000ull;
// A role waits for another through up to two units of the longest context (the walker for the
// tended tiles at a unit's end, while the loader is at its beginning): what a tile may take
// beyond kWaitNs.  A tile takes 2 us when all SMs share the HBM bandwidth.
constexpr uint64_t kWaitNsPerTile = 8192;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;      // log2 of the growth of a row's maximum that P absorbs
// Of 16 pairs of exponentials, those on the FMA pipe.  0, 3, 5 and 8 in turn, 200 calls in a row,
// medians of 15: a 4096-token prompt of 16 heads 101, 96, 94 and 99 us; 512 tokens behind 8K 53.5,
// 51.4, 51.3 and 53.3; 1024 behind 32K, 32 heads, 670, 620, 626 and 661 (spread of one: 3 %).
constexpr int kPoly = 5;
constexpr int kBlock = kKeys * 128;   // bytes of one 64-column block of a 128-row tile

template <int D>
struct Smem {
    static constexpr int TILE = D * 256;                      // a 128-row tile of D bf16 columns
    static constexpr int STAGES = D == 128 ? 5 : 10;          // K and V tiles in flight, in turn
    static constexpr int Q = 0;
    static constexpr int KV = 2 * TILE;
    static constexpr int EXCH = KV + STAGES * TILE;           // the streams' maxima and sums: float [2][2][128]
    static constexpr int BARS = EXCH + 2048;
    static constexpr int SCAN = BARS + 704;                   // the line's scan: a word per warp
    static constexpr int BYTES = SCAN + 8 * (kThreads / 32);
};

// This CTA's part of a unit, handed by the walker to the other roles.
struct Piece {
    int n;                 // key tiles; 0 = the end
    int b, head;           // sequence and key head
    int row0, toks;        // first row of the unit's tokens in q and o, and their number
    int first_pos;         // position of the first one
    int lo, hi;            // keys that some row sees
    int all_lo;            // the first key that the last row sees
    int key0;              // first key of the first tile
    int single;            // one row tile: the streams share it
    int slot;              // where partial results go; -1 = the unit is whole here
    Split split;           // its parts, if it is not
    // the rows [from, to) of tile j that are keys of the unit
    __device__ __forceinline__ int from(int j) const { return max(0, lo - (key0 + j * kKeys)); }
    __device__ __forceinline__ int to(int j) const { return min(kKeys, hi - (key0 + j * kKeys)); }
    // tile j has a key that some row does not see: beyond the first row's position or before
    // the last row's window (which begins at `all_lo`).  Such V tiles go by the walker.
    __device__ __forceinline__ bool tended(int j) const {
        const int k = key0 + j * kKeys;
        return k + kKeys - 1 > first_pos || k < all_lo;
    }
};

struct Bars {
    uint64_t q_full[2], q_free[2], x_full, x_free, drain[2];
    uint64_t s_full[4], p_ready[4], o_step[4];   // per stream and buffer: 2 s + buffer
    uint64_t piece_full[2], piece_free[2];
    uint64_t kv_full[10], kv_free[10];
    uint64_t v_raw[10], v_clean[10];   // tended V tiles: loaded; fit for use
    Piece piece[2];
    int2 dirty[4];         // per piece (counted modulo 4): first and last tile with values replaced, or (.., -1)
    uint32_t tmem;
    int abort;             // a wait ran out
    int bad_page;
    uint64_t limit_ns;     // of a wait for another role
};
static_assert(sizeof(Bars) <= 704, "the barriers fit their space");

struct Maps {
    CUtensorMap q, k, v;
};

// A wait that ends, by one thread: false when it ran out or another role gave up.
__device__ __forceinline__ bool wait_one(Bars* b, uint64_t* bar, uint32_t parity) {
    bool done = mbar_try_wait(bar, parity);
    if (!done) {
        const uint64_t t0 = global_timer_ns();
        while (!(done = mbar_try_wait(bar, parity))) {
            if (*reinterpret_cast<volatile int*>(&b->abort)) break;
            if (global_timer_ns() - t0 > b->limit_ns) {
                *reinterpret_cast<volatile int*>(&b->abort) = 1;   // reported at the end
                break;
            }
        }
    }
    return done;
}

// The same by a whole warp, every lane with the same answer.
__device__ __forceinline__ bool wait(Bars* b, uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_one(b, bar, parity));
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

// The largest of three, NaN if one is: a NaN score makes its row NaN whichever way its
// exponentials are computed.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// 2^y of both halves on the FMA pipe, for y < 128; exactly 0 at and below -127, and for NaN (a
// row with one is NaN by its other exponentials and its offset).  y = n + f
// with n the nearest integer (found by adding 1.5 * 2^23, whose low bits then hold it), 2^f a
// polynomial of degree 5 with value 1 at 0 and else the least relative error on [-1/2, 1/2]
// (a Remez fit of its own: 4.9e-7 in fp32 arithmetic against 2^f in fp64, twice the special
// function unit's error),
// n added to its exponent: -127 leaves none of 1.0's.
__device__ __forceinline__ float2 ex2_poly(Pair y) {
    const float2 in = unpair(y);
    y = pair(fmaxf(in.x, -127.0f), fmaxf(in.y, -127.0f));
    const Pair t = add2(y, pair(12582912.0f, 12582912.0f));
    const Pair n = add2(t, pair(-12582912.0f, -12582912.0f));
    const Pair f = fma2(n, pair(-1.0f, -1.0f), y);
    Pair p = pair(0.0011125507298856974f, 0.0011125507298856974f);
    p = fma2(p, f, pair(0.009666282683610916f, 0.009666282683610916f));
    p = fma2(p, f, pair(0.05557400360703468f, 0.05557400360703468f));
    p = fma2(p, f, pair(0.24022351205348969f, 0.24022351205348969f));
    p = fma2(p, f, pair(0.693142831325531f, 0.693142831325531f));
    p = fma2(p, f, pair(1.0f, 1.0f));
    const float2 e = unpair(p), k = unpair(t);
    return make_float2(__uint_as_float(__float_as_uint(e.x) + (__float_as_uint(k.x) << 23)),
                       __uint_as_float(__float_as_uint(e.y) + (__float_as_uint(k.y) << 23)));
}

// P of a step's scores of one row, 2^(s scale - m scale), as bf16 into 32 TMEM columns; their
// sum is added to sum.  Of 16 pairs, POLY go through the polynomial: the special function
// unit alone (16 results a clock and SM) would need 2048 clocks per 128 keys of both streams.
template <int POLY>
__device__ __forceinline__ void probabilities(const float* x, Pair scale, Pair off, uint32_t to, Pair* sum) {
#pragma unroll
    for (int c = 0; c < kStep / 32; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const Pair y = fma2(pair(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]), scale, off);
            float2 e;
            if ((i * POLY) % 16 < POLY && POLY > 0) {
                e = ex2_poly(y);
            } else {
                e = unpair(y);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
            }
            sum[i & 1] = add2(sum[i & 1], pair(e.x, e.y));
            p[i] = pack(e.x, e.y);
        }
        tmem_st16(to + c * 16, p);
    }
}

// After a wait for TMEM loads: ties 32 loaded values to this point, so that the compiler
// computes nothing with them before it.
__device__ __forceinline__ void loaded32(float* x) {
    asm volatile(""
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]),
                   "+f"(x[6]), "+f"(x[7]), "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]),
                   "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]), "+f"(x[17]),
                   "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]),
                   "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]),
                   "+f"(x[30]), "+f"(x[31]));
}

// Whether rows [r0, r1) of a V tile hold an infinity or a NaN, by a warp: any such value
// times zero is NaN.
template <int D>
__device__ __forceinline__ bool not_finite(uint32_t tile, int r0, int r1) {
    uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int cb = 0; cb < D / 64; ++cb) {
#pragma unroll 4
        for (int i = r0 * 8 + (threadIdx.x & 31); i < r1 * 8; i += 32) {   // 8 pieces of 16 bytes a row
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(tile + cb * kBlock + i * 16)
                         : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc[k]) : "r"(w[k]), "r"(0));
        }
    }
    // every sum is zero (of either sign) or NaN
    const uint32_t any = (acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu;
    return __any_sync(0xffffffffu, any != 0u);
}

// Zeroes what is not finite in a V tile, by a warp.
template <int D>
__device__ __noinline__ void replace_not_finite(uint32_t tile) {
    for (int i = threadIdx.x & 31; i < D * 256 / 4; i += 32) {
        uint32_t w;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(tile + i * 4) : "memory");
        if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
        if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(tile + i * 4), "r"(w) : "memory");
    }
    __syncwarp();
}

// ------------------------------------------------------------------- walker
// Walks this CTA's stretch of the line and hands out its pieces, one ahead of the one in
// work, whose V tiles with keys that some row does not see it tends before the MMA threads
// use them: P is 0 there, but 0 times an infinity or a NaN is not.  Rows outside the unit's
// keys become zero.  Values that are not finite become zero too, and the rows that do see
// them add them at the end; none has been found in a tile after one multiply-add by zero
// per pair of values.
template <int D, typename Seqs>
__device__ __forceinline__ void walk_role(const Args& a, const Line& ln, const Seqs& seqs, uint8_t* smem, Bars* b) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const long long per = ln.per_part;
    const long long start = (long long)blockIdx.x * per, end = min(start + per, ln.total);
    Unit u{};
    bool more = start < end;   // u has tiles in the stretch
    if (more) {
        u = find_unit(a, seqs, start);
        if (start - u.begin >= u.r.tiles) {
            more = unit_end(a, u) < end;
            if (more) next_unit(a, seqs, u);
        }
    }
    unsigned tiles = 0, tended = 0;   // before the piece being tended; parities of v_raw
    Piece last;
    last.n = 0;
    for (unsigned i = 0;; ++i) {
        if (i >= 2 && !wait(b, &b->piece_free[i & 1], (i / 2 - 1) & 1)) return;
        Piece p{};
        if (more) {
            const int kt0 = (int)max(0ll, start - u.begin), kt1 = (int)min((long long)u.r.tiles, end - u.begin);
            p.n = kt1 - kt0;
            p.b = u.b;
            p.head = u.head;
            p.row0 = u.s.row0 + u.r.tok0;
            p.toks = u.r.toks;
            p.first_pos = u.s.ctx - u.s.qlen + u.r.tok0;
            p.lo = u.r.lo;
            p.hi = u.r.hi;
            p.all_lo = first_key(a, p.first_pos + p.toks - 1);
            p.key0 = (u.r.tile0 + kt0) * kKeys;
            p.single = u.r.toks <= a.block_tokens;
            p.slot = p.n == u.r.tiles ? -1 : (int)part_slot(blockIdx.x, u.begin <= start);
            p.split = split_of(u, per);
            more = unit_end(a, u) < end;
        }
        if (lane == 0) {
            b->dirty[i & 3] = make_int2(0, -1);
            b->piece[i & 1] = p;
            mbar_arrive(&b->piece_full[i & 1]);
        }
        __syncwarp();
        if (a.merge_kernel && lane == 0 && !more && p.n > 0 && !p.single && p.slot >= 0 &&
            p.split.first == (int)blockIdx.x && p.split.last > p.split.first)   // the stretch's last piece goes on
            a.splits[blockIdx.x] = SplitUnit{p.split.last, p.split.from_start, p.row0, p.toks, p.head, p.first_pos, {}};
        for (int j = 0; j < last.n; ++j, ++tiles) {
            if (!last.tended(j)) continue;
            const int from = last.from(j), to = last.to(j);
            const unsigned st = (2 * tiles + 1) % S::STAGES;
            if (!wait(b, &b->v_raw[st], (tended >> st) & 1)) return;
            tended ^= 1u << st;
            const uint32_t tile = base + S::KV + st * S::TILE;
            if (from > 0 || to < kKeys) {
                for (int r = lane; r < kKeys * (D / 64); r += 32) {
                    if (r % kKeys >= from && r % kKeys < to) continue;
                    const uint32_t row = tile + (r / kKeys) * kBlock + (r % kKeys) * 128;
#pragma unroll
                    for (int c = 0; c < 128; c += 16)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + c), "r"(0) : "memory");
                }
                __syncwarp();
            }
            // the keys that some row sees and some row does not: before the last row's window,
            // and beyond the first row's position
            const int key0 = last.key0 + j * kKeys;
            const int before = min(to, last.all_lo - key0), beyond = max(from, last.first_pos + 1 - key0);
            if (last.toks > 1 && (not_finite<D>(tile, from, before) || not_finite<D>(tile, beyond, to))) {
                replace_not_finite<D>(tile);
                if (lane == 0) {
                    int2& d = b->dirty[(i - 1) & 3];
                    d = make_int2(d.y < 0 ? j : d.x, j);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->v_clean[st]);
        }
        last = p;
        if (p.n == 0) return;
        if (more) next_unit(a, seqs, u);
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
    __device__ __forceinline__ Piece get_one(Bars* b) {   // for a single thread
        Piece p;
        p.n = 0;
        if (wait_one(b, &b->piece_full[i & 1], (i / 2) & 1)) p = b->piece[i & 1];
        mbar_arrive(&b->piece_free[i & 1]);
        ++i;
        return p;
    }
};

// Which of the two Q tiles a piece has, and how often each was used before: a piece of two
// row tiles has both, single ones take turns, so that the next one's Q is loaded ahead.  The
// loader and the MMA threads count alike.
struct QTiles {
    unsigned uses[2] = {0, 0};
    int turn = 0;
    __device__ __forceinline__ bool has(const Piece& p, int t) const { return !p.single || t == turn; }
    __device__ __forceinline__ void next(const Piece& p) {
        if (has(p, 0)) ++uses[0];
        if (has(p, 1)) ++uses[1];
        if (p.single) turn ^= 1;
    }
};

// ------------------------------------------------------------------- loader
template <int D>
__device__ __forceinline__ void load_role(const Args& a, const Maps& maps, uint8_t* smem, Bars* b, int granule) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const int runs = kKeys / granule;           // TMA boxes of one 64-column block
    unsigned ring = 0, raws = 0, raw_any = 0;   // raws: parities of v_raw
    unsigned q_loads[2] = {0, 0};
    QTiles qt;
    bool ok = true;
    Pieces pieces;
    for (Piece u = pieces.get(b); u.n > 0; u = pieces.get(b)) {
        // Q, once the scores of the last piece that had the tile are done with it
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (!qt.has(u, t)) continue;
            ok = ok && (qt.uses[t] == 0 || wait(b, &b->q_free[t], (qt.uses[t] - 1) & 1));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&b->q_full[t], (uint32_t)(D * 2 * a.group * a.block_tokens));
            __syncwarp();
            if (lane < D / 64)
                tma_load_3d(smem + S::Q + t * S::TILE + lane * kBlock, &maps.q, &b->q_full[t], lane * 64, u.head * a.group,
                            u.row0 + (u.single ? 0 : t * a.block_tokens));
            ++q_loads[t];
        }
        if (!ok) break;
        qt.next(u);
        // this lane's run of rows of a tile and its page number, read a tile ahead: past the
        // pool (read as zeros) when the run holds no key of the unit
        const int run = lane % runs;
        auto page_of = [&](int j) {
            const int key = u.key0 + j * kKeys + run * granule;
            return j < u.n && key < u.hi && key + granule > u.lo
                       ? a.page_table[(long long)u.b * a.max_pages + key / a.page_size]
                       : a.num_pages;
        };
        int next_page = page_of(0);
        for (int j = 0; ok && j < u.n; ++j) {
            const int key = u.key0 + j * kKeys + run * granule;
            int page = next_page;
            next_page = page_of(j + 1);
            if (page < 0 || page >= a.num_pages) {   // a bad number reads as zeros too, and is reported
                if (key < u.hi && key + granule > u.lo) *reinterpret_cast<volatile int*>(&b->bad_page) = 1;
                page = a.num_pages;
            }
            const int in_page = key % a.page_size;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const unsigned st = ring % S::STAGES, ph = ring / S::STAGES;
                ok = ph == 0 || wait(b, &b->kv_free[st], (ph - 1) & 1);
                if (!ok) break;
                // a ragged V tile goes to the walker first; its own phase then passes empty
                const bool raw = kv == 1 && u.tended(j);
                uint64_t* full = raw ? &b->v_raw[st] : &b->kv_full[st];
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, S::TILE);
                    if (raw) mbar_arrive(&b->kv_full[st]);
                }
                if (raw) raws ^= 1u << st, raw_any |= 1u << st;
                __syncwarp();
                // a lane per (column block, run); 32 is a multiple of the runs, so a lane's run is its own
                for (int i = lane; i < runs * (D / 64); i += 32) {
                    const int cb = i / runs;
                    tma_load_4d(base + S::KV + st * S::TILE + cb * kBlock + run * granule * 128,
                                kv == 0 ? &maps.k : &maps.v, full, cb * 64, u.head, in_page, page);
                }
                __syncwarp();
                ++ring;
            }
        }
    }
    // This warp's copies are in before the CTA may leave, whichever way the loop ended: another
    // role may give up, now or later, with some of them on their way.  (The products wait for
    // the same copies, so this delays nothing.)
    const unsigned n = min(ring, (unsigned)S::STAGES);
    for (unsigned i = ring - n; i < ring; ++i) mbar_wait_bounded(&b->kv_full[i % S::STAGES], (i / S::STAGES) & 1, kWaitNs);
    for (int i = 0; i < S::STAGES; ++i)
        if ((raw_any >> i) & 1) mbar_wait_bounded(&b->v_raw[i], ((raws >> i) & 1) ^ 1, kWaitNs);
    for (int t = 0; t < 2; ++t)
        if (q_loads[t]) mbar_wait_bounded(&b->q_full[t], (q_loads[t] - 1) & 1, kWaitNs);
}

// --------------------------------------------------------------- MMA issuers
// One thread per stream issues its products, in the order QK(h + 1), PV(h): the scores of a
// step are computed while the softmax of the step before runs.  A warp for both streams,
// with its waits and elections, took 2560 clocks a step, twice the tensor core's time.
template <int D>
__device__ __forceinline__ void mma_role(const Args& a, uint8_t* smem, Bars* b, int s) {
    using S = Smem<D>;
    const uint32_t base = smem_u32(smem), tm = b->tmem;
    const uint32_t id_s = idesc_bf16(128, kStep, false, false), id_o = idesc_bf16(128, D, false, true);
    unsigned tiles = 0, steps = 0, cleaned = 0;   // before this piece; parities of v_clean
    QTiles qt;
    bool ok = true;
    Pieces pieces;
    for (Piece u = pieces.get_one(b); u.n > 0; u = pieces.get_one(b)) {
        // steps: single: step h is tile h, half s; else tile h / 2, half h % 2
        const bool single = u.single;
        const int H = single ? u.n : 2 * u.n;
        const int q = single ? qt.turn : s;   // this stream's Q tile
        const uint64_t dq = smem_desc_sw128(base + S::Q + q * S::TILE, 16, 1024);
        // S of step h into its buffer, over the P of step h - 2, whose product has to be
        // complete: products into different accumulators are not ordered by their issue
        auto scores = [&](int h) {
            const unsigned G = steps + h, buf = G & 1, at = 2 * (tiles + (single ? h : h >> 1)), st = at % S::STAGES;
            const int half = single ? s : h & 1;
            if (single || half == 0) ok = wait_one(b, &b->kv_full[st], (at / S::STAGES) & 1);
            if (ok && G >= 2) ok = wait_one(b, &b->o_step[2 * s + buf], ((G - 2) >> 1) & 1);
            if (!ok) return;
            tc_fence_after();
            const uint64_t dk = smem_desc_sw128(base + S::KV + st * S::TILE + half * (kStep * 128), 16, 1024);
            const uint32_t d = tm + s * 128 + buf * 64;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kBlock + (kk & 3) * 32;
                mma_bf16_ss(d, desc_advance(dq, off), desc_advance(dk, off), id_s, kk > 0);
            }
            mma_commit(&b->s_full[2 * s + buf]);
            if (single || half == 1) mma_commit(&b->kv_free[st]);
            if (h == H - 1) {   // two arrivals a tile: each stream is done with every tile of the piece
                if (qt.has(u, 0)) mma_commit(&b->q_free[0]);
                if (qt.has(u, 1)) mma_commit(&b->q_free[1]);
            }
        };
        ok = wait_one(b, &b->q_full[q], (q ? qt.uses[1] : qt.uses[0]) & 1);
        if (ok) scores(0);
        for (int h = 0; ok && h < H; ++h) {
            if (h + 1 < H) scores(h + 1);
            if (!ok) break;
            const unsigned G = steps + h, buf = G & 1, at = 2 * (tiles + (single ? h : h >> 1)) + 1, st = at % S::STAGES;
            const int half = single ? s : h & 1;
            if (single || half == 0) {
                if (u.tended(single ? h : h >> 1)) {   // the walker's word that it is clean
                    ok = wait_one(b, &b->v_clean[st], (cleaned >> st) & 1);
                    cleaned ^= 1u << st;
                } else {
                    ok = wait_one(b, &b->kv_full[st], (at / S::STAGES) & 1);
                }
            }
            if (ok) ok = wait_one(b, &b->p_ready[2 * s + buf], (G >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dv = smem_desc_sw128(base + S::KV + st * S::TILE + half * (kStep * 128), kBlock, 1024);
            const uint32_t d = tm + 256 + s * 128, p = tm + s * 128 + buf * 64;
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)
                mma_bf16_ts(d, p + kk * 8, desc_advance(dv, kk * 2048), id_o, h > 0 || kk > 0);
            mma_commit(&b->o_step[2 * s + buf]);
            if (single || half == 1) mma_commit(&b->kv_free[st]);
        }
        if (!ok) break;
        tiles += u.n;
        steps += H;
        qt.next(u);
    }
    // everything issued is complete before the TMEM goes back
    mma_commit(&b->drain[s]);
    mbar_wait_bounded(&b->drain[s], 0, kWaitNs);
}

// ---------------------------------------------------------------- the merge
// A warp's rows of a split unit merged from its parts: a lane has one row (lse_row of the
// log-sums) and of its columns the groups of four first, first + step, ...; group g of a part
// sits at offset + g * stride values in the part's slot.  The latency of the reads is most of
// the cost, so PARTS parts of GROUPS groups are read at once, their log-sums beside them.
template <int D>
struct Merge {
    const Args& a;
    const Split& sp;
    int lse_row;
    long long offset;
    int stride;
    bool mine;                // the lane has a row
    bool sees;                // and that sees a key
    int groups, first, step;

    template <int GROUPS, int PARTS>
    __device__ __forceinline__ void run(__nv_bfloat16* to, float* lse_out) const {
        for (int g0 = first; g0 < groups; g0 += GROUPS * step) {
            float top = -INFINITY, sum = 0.0f;
            float4 acc[GROUPS];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) acc[g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int p0 = sp.first; p0 <= sp.last; p0 += PARTS) {
                float w[PARTS];
                float4 y[PARTS][GROUPS];
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    const bool on = mine && p0 + i <= sp.last;
                    const long long slot = on ? sp.slot(p0 + i) : 0;
                    w[i] = on ? __ldcg(a.part_lse + slot * (2 * kRows) + lse_row) : -INFINITY;
                    const float* from = a.part_o + slot * (2 * kRows * D) + offset;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g)
                        y[i][g] = on && g0 + g * step < groups
                                      ? __ldcg(reinterpret_cast<const float4*>(from + (g0 + g * step) * stride))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                float t = top;
#pragma unroll
                for (int i = 0; i < PARTS; ++i) t = fmaxf(t, w[i]);
                const float ref = t == -INFINITY ? 0.0f : t, keep = ex2(top - ref);
                top = t;
                sum *= keep;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    acc[g].x *= keep;
                    acc[g].y *= keep;
                    acc[g].z *= keep;
                    acc[g].w *= keep;
                }
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    const float f = ex2(w[i] - ref);
                    sum += f;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        acc[g].x = fmaf(f, y[i][g].x, acc[g].x);
                        acc[g].y = fmaf(f, y[i][g].y, acc[g].y);
                        acc[g].z = fmaf(f, y[i][g].z, acc[g].z);
                        acc[g].w = fmaf(f, y[i][g].w, acc[g].w);
                    }
                }
            }
            const float inv = inverse_sum(sum, sees);   // a NaN part makes the row NaN
            if (lse_out && g0 == 0) *lse_out = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
                if (mine && g0 + g * step < groups)
                    *reinterpret_cast<uint2*>(to + 4 * (g0 + g * step)) =
                        make_uint2(pack(acc[g].x * inv, acc[g].y * inv), pack(acc[g].z * inv, acc[g].w * inv));
        }
    }
};

// ------------------------------------------------------------ softmax groups
// The lanes whose bit BIT of the lane number is 0 give their y and the others their x to the
// lane across.
template <int BIT>
__device__ __forceinline__ void trade(uint32_t (&x)[4], uint32_t (&y)[4]) {
    const bool upper = threadIdx.x & BIT;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[i] : y[i], BIT);
        if (upper) x[i] = got;
        else y[i] = got;
    }
}

template <int D>
__device__ __forceinline__ void softmax_role(const Args& a, uint8_t* smem, Bars* b, int s) {
    using S = Smem<D>;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tm = b->tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tm_o = tm + 256 + s * 128;
    float* exch = reinterpret_cast<float*>(smem + S::EXCH);
    const float sl = a.scale * 1.4426950408889634f;
    const int row_tok = row / a.group, row_head = row % a.group;   // of a row tile's rows
    unsigned steps = 0, x_count = 0;   // steps of this stream, over all pieces
    bool ok = true;
    Pieces pieces;
    for (Piece u = pieces.get(b); u.n > 0; u = pieces.get(b)) {
        const int sub = u.single ? 0 : s;
        const int toks = min(a.block_tokens, u.toks - sub * a.block_tokens);
        const int rows = toks * a.group;
        const int first_pos = u.first_pos + sub * a.block_tokens;
        const int top_key = row < rows ? first_pos + row_tok : -1;     // keys [low_key, top_key] are seen
        const int low_key = first_key(a, top_key);
        // keys that every row of the tile sees: [all_lo, all_hi]
        const int all_hi = first_pos;
        const int all_lo = first_key(a, first_pos + toks - 1);
        const bool active = quarter * 32 < rows;   // this warp has rows
        // while the first scores are on their way
        const bool counted =
            active && u.slot >= 0 && u.single && lane == 0 && claim_arrivals(a, u.split, s * 4 + quarter);
        __syncwarp();
        float m = -INFINITY;
        const Pair scale = pair(sl, sl);
        Pair sum[2] = {0ull, 0ull};
        const int H = u.single ? u.n : 2 * u.n;
        for (int h = 0; h < H; ++h, ++steps) {
            const unsigned buf = steps & 1;
            const uint32_t tm_s = tm + s * 128 + buf * 64;
            ok = wait(b, &b->s_full[2 * s + buf], (steps >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (active) {
                const int key0 = u.key0 + (u.single ? 2 * h + s : h) * kStep;
                float x[kStep];
                tmem_ld32(tm_s, x);
                tmem_ld32(tm_s + 32, x + 32);
                tmem_wait_ld();
                loaded32(x);
                loaded32(x + 32);
                const bool masked = key0 < all_lo || key0 + kStep - 1 > all_hi;
                if (masked) {
                    // the keys of the step that this row sees, a bit each
                    const int end = top_key - key0 + 1, begin = low_key - key0;
                    const unsigned long long seen =
                        (end >= kStep ? ~0ull : end <= 0 ? 0ull : (1ull << end) - 1) &
                        (begin <= 0 ? ~0ull : begin >= kStep ? 0ull : ~0ull << begin);
#pragma unroll
                    for (int i = 0; i < kStep; ++i) x[i] = (seen >> i) & 1 ? x[i] : -INFINITY;
                }
                float t0 = max3(m, x[0], x[1]), t1 = max3(x[2], x[3], x[4]), t2 = max3(x[5], x[6], x[7]);
#pragma unroll
                for (int i = 8; i < 62; i += 6) {
                    t0 = max3(t0, x[i], x[i + 1]);
                    t1 = max3(t1, x[i + 2], x[i + 3]);
                    t2 = max3(t2, x[i + 4], x[i + 5]);
                }
                t0 = max3(t0, x[62], x[63]);
                const float top = max3(t0, t1, t2);
                // also when a NaN came in; not when all is still masked, nor for rows that are
                // no rows.  Each row decides for itself: what shares its warp changes no bit of it.
                const bool grown = row < rows && !((top - m) * sl <= kLazy) && top != -INFINITY;
                if (__any_sync(0xffffffffu, grown)) {
                    const float f = !grown ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - top) * sl);
                    sum[0] = fma2(sum[0], pair(f, f), 0ull);
                    sum[1] = fma2(sum[1], pair(f, f), 0ull);
                    m = grown ? top : m;
                    if (h > 0) {   // the last product into O, if it is not complete yet
                        ok = wait(b, &b->o_step[2 * s + (buf ^ 1)], ((steps - 1) >> 1) & 1);
                        tc_fence_after();
#pragma unroll 1   // small, beside the hot path
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
                // An infinite maximum (a score of +infinity, or finite ones beyond fp32 once scaled)
                // has no softmax: 0 x off makes the offset, and so every exponential of the row, NaN.
                // The polynomial's clamp would turn the NaN of infinity - infinity into 0.
                float off = m == -INFINITY ? 0.0f : -m * sl;
                off = fmaf(off, 0.0f, off);
                probabilities<kPoly>(x, scale, pair(off, off), tm_s, sum);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->p_ready[2 * s + buf]);
        }
        const float2 sums = unpair(add2(sum[0], sum[1]));
        const float l = sums.x + sums.y;
        if (ok) ok = wait(b, &b->o_step[2 * s + ((steps - 1) & 1)], ((steps - 1) >> 1) & 1);
        if (!ok) break;
        if (u.single) {   // both streams' outputs are complete, their maxima and sums exchanged
            exch[s * 256 + row] = m;
            exch[s * 256 + 128 + row] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->x_full);
            ok = wait(b, &b->x_full, x_count & 1);
            if (!ok) break;
        }
        tc_fence_after();
        const long long orow =
            (long long)(u.row0 + sub * a.block_tokens + row_tok) * a.num_heads + u.head * a.group + row_head;
        const bool whole = u.slot < 0;
        const int2 dirty = b->dirty[(pieces.i - 1) & 3];
        // Partial outputs of this warp's rows (single: of this group's half of their columns):
        // [columns / 4][R] float4 with R the rows of the warp, rounded up to a power of two, so
        // that both the writes (a lane per row) and the merge's reads are of whole lines.
        const int warp_rows = min(32, rows - quarter * 32);
        const int log_r = warp_rows <= 1 ? 0 : 32 - __clz(warp_rows - 1), R = 1 << log_r;
        const long long warp_at = (long long)(s * 4 + quarter) * 32 * (u.single ? D / 2 : D);   // in a slot
        if (active) {
            // weights of the two streams' sums (the other stream has other rows: 0)
            float f0 = 1.0f, f1 = 0.0f, sum = l, top = m;
            if (u.single) {
                const float m0 = exch[row], l0 = exch[128 + row], m1 = exch[256 + row], l1 = exch[256 + 128 + row];
                top = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.0f : ex2((m0 - top) * sl);
                f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - top) * sl);
                sum = l0 * f0 + l1 * f1;
            }
            const float inv = inverse_sum(sum, whole && top_key >= 0);
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
                if (u.single) {
                    float z[32];
                    tmem_ld32(from + 128 + c * 32, z);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(z[i], f1, o[i]);
                }
                if (__builtin_expect(dirty.y >= 0, 0)) {
                    // the values that the walker replaced, for the rows that see them
                    const int k0 = max(max(low_key, u.lo), u.key0 + dirty.x * kKeys);
                    const int k1 = min(min(top_key + 1, u.hi), u.key0 + (dirty.y + 1) * kKeys);
#pragma unroll 1
                    for (int key = k0; key < k1; ++key) {
                        if (!u.tended((key - u.key0) / kKeys)) continue;
                        const int page = a.page_table[(long long)u.b * a.max_pages + key / a.page_size];
                        if (page < 0 || page >= a.num_pages) continue;
                        const uint32_t* v = reinterpret_cast<const uint32_t*>(
                            static_cast<const __nv_bfloat16*>(a.v) + (long long)page * a.page_stride +
                            (long long)(key % a.page_size) * a.row_stride + (long long)u.head * a.head_stride + c * 32);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t w = v[i];
                            if ((w & 0x7f80u) == 0x7f80u) o[2 * i] += __uint_as_float(w << 16);
                            if ((w & 0x7f800000u) == 0x7f800000u) o[2 * i + 1] += __uint_as_float(w & 0xffff0000u);
                        }
                    }
                }
                if (whole) {
                    // four lanes trade their rows' 16-byte pieces, so that they store 64 bytes of
                    // one row at a time (a lane per row: 32 lines a store, 4 us a unit)
                    uint32_t w[4][4];   // [piece of my row], then [row of the four][word of piece lane % 4]
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = pack(o[2 * i], o[2 * i + 1]);
                    trade<1>(w[0], w[1]);
                    trade<1>(w[2], w[3]);
                    trade<2>(w[0], w[2]);
                    trade<2>(w[1], w[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const long long to = __shfl_sync(0xffffffffu, orow, (lane & ~3) + i);
                        if (quarter * 32 + (lane & ~3) + i < rows)
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + to * D + c * 32 + (lane & 3) * 8) =
                                make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                    }
                } else if (row < rows) {
                    float4* to = reinterpret_cast<float4*>(a.part_o + (long long)u.slot * (2 * kRows * D) + warp_at) +
                                 (c - c0) * 8 * R + lane;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        to[i * R] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (row < rows) {
                const float lse2 = sum == 0.0f ? -INFINITY : top * sl + log2f(sum);
                // each group keeps a copy with its share of the outputs
                if (!whole) a.part_lse[(long long)u.slot * (2 * kRows) + s * kRows + row] = lse2;
                else if (a.lse && (!u.single || s == 0)) a.lse[orow] = lse2 * kLn2;
            }
            if (!whole && u.single) {
                // the warp that brings the last part of its half of its rows' columns merges them
                __threadfence();
                __syncwarp();
                const bool last = __shfl_sync(0xffffffffu, counted && arrive_last(a, u.split, s * 4 + quarter), 0);
                if (last) {
                    const int r = lane & (R - 1), at = quarter * 32 + r;
                    const long long orow_r = __shfl_sync(0xffffffffu, orow, r);
                    const Merge<D> mg{a, u.split, s * kRows + at, warp_at + 4 * r, 4 * R, at < rows,
                                      first_pos + at / a.group >= 0, D / 8, lane >> log_r, 32 >> log_r};
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.o) + orow_r * D + s * (D / 2);
                    float* lse = a.lse && at < rows && lane < R && s == 0 ? a.lse + orow_r : nullptr;
                    // few rows have few columns a lane, so as many more parts in flight (20 parts of 4
                    // rows, 6 and 10 at a time: 6.2 and 3.9 us)
                    if (R <= 4) mg.template run<2, 10>(to, lse);
                    else mg.template run<4, 6>(to, lse);
                }
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
    Line ln;
    if (a.merge_kernel && threadIdx.x == 0) a.splits[blockIdx.x].last = -1;   // until the walker knows better
    if (a.line_inline != 2) {
        ln = get_line<kThreads>(a, reinterpret_cast<long long*>(smem + S::SCAN));
        if ((int)blockIdx.x >= ln.parts) return;
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.ws->epoch = a.epoch;
    }
    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the runtime places the block's memory so
        if (threadIdx.x == 0) tag_merge_inline(&a.ws->status, a.epoch, kStatusBounds, false);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(&b->x_full, 8);
        mbar_init(&b->x_free, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&b->q_full[s], 1);
            mbar_init(&b->q_free[s], 2);
            mbar_init(&b->piece_full[s], 1);
            mbar_init(&b->piece_free[s], 11);   // the softmax and MMA warps, the loader
            mbar_init(&b->drain[s], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&b->s_full[i], 1);
            mbar_init(&b->p_ready[i], 4);
            mbar_init(&b->o_step[i], 1);
        }
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&b->kv_full[i], 1);
            mbar_init(&b->kv_free[i], 2);       // both streams
            mbar_init(&b->v_raw[i], 1);
            mbar_init(&b->v_clean[i], 1);
        }
        b->abort = b->bad_page = 0;
        b->limit_ns = kWaitNs + kWaitNsPerTile * (min((long long)kMostKeys, (long long)a.max_pages * a.page_size) / kKeys);
        mbar_fence_init();
    }
    if (warp == 8) {
        tmem_alloc(&b->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 10 && elect_one()) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < 8) {
        softmax_role<D>(a, smem, b, warp >> 2);
    } else if (warp < 10) {
        if (elect_one()) mma_role<D>(a, smem, b, warp - 8);
        __syncwarp();
    } else if (warp == 10) {
        load_role<D>(a, maps, smem, b, granule);
    } else {
        if (a.line_inline == 2) {
            LaneSeqs seqs{a};
            ln = lane_line(a, seqs);
            walk_role<D>(a, ln, seqs, smem, b);
        } else {
            walk_role<D>(a, ln, StoredSeqs{a}, smem, b);
        }
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

// The units of two row tiles that the cuts split, each by its parts in the order of the
// line: block (i, share) the unit that CTA i of the attention kernel began, 32 rows of it, the
// columns over eight warps.  At most 38 MB of parts (two a CTA), read once by
// all SMs.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const SplitUnit u = a.splits[blockIdx.x];
    if (!to_merge(u, blockIdx.x, a.shape.max_parts, a.block_tokens * a.shape.subs, a.rows, a.num_kv_heads)) return;
    const int s = blockIdx.y >> 2, quarter = blockIdx.y & 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(a.block_tokens, u.toks - s * a.block_tokens) * a.group;
    const int warp_rows = min(32, rows - quarter * 32);
    if (warp_rows <= 0) return;
    const int log_r = warp_rows <= 1 ? 0 : 32 - __clz(warp_rows - 1), R = 1 << log_r;
    const int r = lane & (R - 1), at = quarter * 32 + r;
    const long long row = (long long)(u.row0 + s * a.block_tokens + at / a.group) * a.num_heads + u.head * a.group +
                          at % a.group;
    const Split sp{(int)blockIdx.x, u.last, u.from_start != 0};
    const int step = 32 >> log_r;
    const Merge<D> mg{a, sp, s * kRows + at, (long long)(s * 4 + quarter) * 32 * D + 4 * r, 4 * R, at < rows,
                      u.first_pos + s * a.block_tokens + at / a.group >= 0, D / 4, (lane >> log_r) + warp * step, 8 * step};
    float* lse = a.lse && at < rows && lane < R && warp == 0 ? a.lse + row : nullptr;
    mg.template run<4, 6>(static_cast<__nv_bfloat16*>(a.o) + row * D, lse);
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
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess || !a.merge_kernel) return launched;
    return launch_merge(merge_kernel<D>, dim3(kMaxParts - 1, 8), a, stream);
}

}  // namespace

// unit_extra 2 (a unit's start and output, beside tiles of about 2 us): a prompt of 4096 tokens
// and 32 chunks of new tokens took 127 and 34 us with 0, 93 and 31 with 2, 93 and 35 with 6.
Shape shape_tc() { return Shape{kRows, 2, kKeys, kMaxParts, kThreads, 2, 2, 0}; }

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
