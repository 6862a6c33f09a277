// gdn_attn.h -- paged attention: the call's arguments and the schedule that its kernels
// share.  Not part of the public ABI.
//
// The work is cut by key tiles.  A unit is a block of consecutive new tokens of one
// sequence with the query heads of one key head (rows = tokens x heads of the group);
// its length is the number of key tiles that its causal (and window) range touches, and
// unit_extra more at its end for what a unit costs beside its tiles.  The units, in the
// order (sequence, key head, token block), form one line of length `total`, and each of
// `parts` CTAs takes the same length of it, wherever units begin and end.  So one long
// context with one new token and a thousand short ones both fill the GPU.  (Without the
// extra, the CTAs with a prompt's short first blocks took 115 us where others took 75.)
//
// A CTA that holds a unit whole writes its outputs.  A unit that the cuts split leaves
// normalised partial outputs and log-sums; whoever brings the last part of some rows
// merges all of them, in the order of the line, so the result does not depend on which
// CTA that was.  Units of many rows (bf16: two row tiles; fp32: more than 8 rows) are
// merged by a kernel of their own, over all SMs: their parts, up to 128 KB each, took the
// last CTA 12 to 15 us.
//
// The lengths are read on the device (a captured call may be replayed with new ones).
// When the sequences and their token blocks are few, every CTA lays out the line for
// itself as it starts; otherwise a one-block kernel does it first.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_hybrid.h"

namespace gdn {
namespace attn {

constexpr int kMostKeys = 1 << 30;   // of a context: sums of positions and tile sizes stay in an int
constexpr int kArrivals = 8;     // separately merged shares of a split unit's rows, at most

// One sequence of the line, 32 bytes.
struct Seq {
    int row0;            // first row of its new tokens in q and o
    int qlen;            // new tokens; 0 if its descriptor entries are bad
    int ctx;             // context length, the new tokens included
    int pad;
    long long head_len;  // length of one key head's units on the line
    long long before;    // length of the sequences before it
};
static_assert(sizeof(Seq) == 32, "Seq is 32 bytes");

// The line, in the workspace after the status header.
struct Line {
    long long total;
    long long per_part;  // length of each CTA's stretch (the last may have less)
    int parts;           // CTAs with work
    int pad[59];
};
static_assert(sizeof(Line) == 256, "Line is 256 bytes");

// A unit of many rows that begins in CTA i and ends in a later one, for the merging kernel:
// slot i of a table that every CTA writes, "none" as it starts and the unit once it has
// handed that out: a CTA that gives up leaves no entry of an earlier call, and no bytes that
// the workspace happened to hold.
struct SplitUnit {
    int last;            // its last part; -1 = there is no such unit
    int from_start;      // it begins where CTA i's stretch does
    int row0, toks, head;
    int first_pos;       // position of its first token
    int pad[2];
};
static_assert(sizeof(SplitUnit) == 32, "SplitUnit is 32 bytes");

// Whether slot i of the table is a unit to be merged: what the merging kernel reads (parts of
// `parts` CTAs) and writes (rows of o) by it then lies within the call's extents.
__host__ __device__ inline bool to_merge(const SplitUnit& u, int i, int parts, int most_toks, long long rows,
                                         int num_kv_heads) {
    return u.last > i && u.last < parts && u.toks > 0 && u.toks <= most_toks && u.row0 >= 0 &&
           (long long)u.row0 + u.toks <= rows && u.head >= 0 && u.head < num_kv_heads;
}

// Sizes that a kernel family fixes.
struct Shape {
    int sub_rows;        // rows of one row tile
    int subs;            // row tiles of a unit
    int tile_keys;       // keys of a tile
    int max_parts;       // CTAs of the grid
    int threads;         // of a CTA
    int min_tiles;       // least length of a CTA's stretch, so that splitting pays
    int unit_extra;      // a unit's cost beside its tiles, in tiles
    int few_rows;        // rows of a unit that its last part's CTA merges (one row tile per unit only)
};

struct Args {
    int dtype, batch, num_heads, num_kv_heads, group, dim;
    int page_size, num_pages, max_pages;    // max_pages: entries per row of the page table
    int block_tokens;                       // tokens of a row tile: sub_rows / group
    Shape shape;
    long long rows;                         // rows of q and o
    long long rs_q;
    long long page_stride, row_stride, head_stride;
    float scale;                            // of the scores
    int window;                             // keys that a row sees at most; 0 = all
    const void* q;
    const void* k;
    const void* v;
    const int* page_table;                  // [batch, max_pages]
    const int* cu;                          // [batch + 1]
    const int* ctx;                         // [batch]
    void* o;                                // [rows, num_heads, dim] packed
    float* lse;                             // [rows, num_heads] or null
    WorkspaceHeader* ws;
    unsigned int epoch;
    int line_inline;                        // every CTA lays out the line itself; 2: each of its warps that needs it
    Line* line;
    Seq* seqs;                              // [batch]
    unsigned long long* arrivals;           // [max_parts * kArrivals]: parts of split units that are in
    int merge_kernel;                       // there may be units that the merging kernel merges
    SplitUnit* splits;                      // [max_parts]
    float* part_lse;                        // [2 * max_parts][subs * sub_rows], base 2
    float* part_o;                          // [2 * max_parts] slots of subs * sub_rows * dim values
};

// What a row's outputs are multiplied by, given the sum of its weights.  A row that sees no key
// has the sum 0 and gets zeros; one that sees keys has it only if every score is -infinity, and
// such a row has no softmax.  Parts decide nothing: `sees` is for
// whole rows and merged ones.
__device__ __forceinline__ float inverse_sum(float sum, bool sees) {
    return sum != 0.0f ? 1.0f / sum : sees ? __int_as_float(0x7fffffff) : 0.0f;   // a NaN sum stays
}

__device__ __forceinline__ void report(const Args& a, unsigned int bits) {
    tag_merge(&a.ws->status, a.epoch, bits, false);
}

// The key range and tiles of token block t of a sequence.
struct Range {
    int tok0, toks;      // first new token of the block and their number
    int lo, hi;          // keys seen by at least one of its rows: [lo, hi)
    int tile0, tiles;    // key tiles; at least one, so that rows without keys are written too
};

// The first key that a row sees which sees none after `top` (which may be negative).
__device__ __forceinline__ int first_key(const Args& a, int top) {
    return a.window > 0 && top >= a.window ? top - a.window + 1 : 0;
}

__device__ __forceinline__ Range block_range(const Args& a, int qlen, int ctx, int t) {
    Range r;
    const int step = a.block_tokens * a.shape.subs;
    r.tok0 = t * step;
    r.toks = min(step, qlen - r.tok0);
    const int first = ctx - qlen + r.tok0;           // position of the first row (may be negative)
    r.hi = max(0, first + r.toks);
    r.lo = min(first_key(a, first), r.hi);
    r.tile0 = r.lo / a.shape.tile_keys;
    r.tiles = max(1, (r.hi + a.shape.tile_keys - 1) / a.shape.tile_keys - r.tile0);
    return r;
}

__device__ __forceinline__ int token_blocks(const Args& a, int qlen) {
    const int step = a.block_tokens * a.shape.subs;
    return (qlen + step - 1) / step;
}

// A unit and its place on the line.
struct Unit {
    int b, head, t;      // sequence, key head, token block
    Range r;
    Seq s;
    long long begin;     // where it begins on the line
};

// The sequences of the line as find_unit and next_unit see them, for a whole warp: in the
// workspace, or (at most 32) one per lane.
struct StoredSeqs {
    const Args& a;
    __device__ __forceinline__ Seq get(int b) const { return a.seqs[b]; }
    // the last sequence with before <= pos
    __device__ __forceinline__ int find(long long pos) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = a.batch;                    // it is in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int i = lo + lane * step;
            const bool below = i < hi && a.seqs[i].before <= pos;
            const int n = __popc(__ballot_sync(0xffffffffu, below));   // lane 0 is always below
            lo = lo + (n - 1) * step;
            hi = min(hi, lo + step);
        }
        return lo;
    }
};
struct LaneSeqs {
    const Args& a;
    Seq mine;
    __device__ __forceinline__ Seq get(int b) const {
        Seq s;
        s.row0 = __shfl_sync(0xffffffffu, mine.row0, b);
        s.qlen = __shfl_sync(0xffffffffu, mine.qlen, b);
        s.ctx = __shfl_sync(0xffffffffu, mine.ctx, b);
        s.pad = 0;
        s.head_len = __shfl_sync(0xffffffffu, mine.head_len, b);
        s.before = __shfl_sync(0xffffffffu, mine.before, b);
        return s;
    }
    __device__ __forceinline__ int find(long long pos) const {
        return 31 - __clz(__ballot_sync(0xffffffffu, (int)(threadIdx.x & 31) < a.batch && mine.before <= pos));
    }
};

// The unit that holds place `pos` of the line (0 <= pos < total), by a whole warp.
template <typename Seqs>
__device__ __forceinline__ Unit find_unit(const Args& a, const Seqs& seqs, long long pos) {
    const int lane = threadIdx.x & 31;
    Unit u;
    u.b = seqs.find(pos);
    u.s = seqs.get(u.b);
    const long long in = pos - u.s.before;
    u.head = ((in | u.s.head_len) >> 32) ? (int)(in / u.s.head_len)
                                           : (int)((uint32_t)in / (uint32_t)u.s.head_len);
    const long long rem = in - u.head * u.s.head_len;
    const int blocks = token_blocks(a, u.s.qlen);
    long long done = 0;
    for (int t0 = 0;; t0 += 32) {                    // ends: rem < head_len = the sum over all blocks
        const int t = t0 + lane;
        const int n = t < blocks ? block_range(a, u.s.qlen, u.s.ctx, t).tiles + a.shape.unit_extra : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, done + incl > rem);
        if (hit || t0 + 32 >= blocks) {
            const int l = hit ? __ffs(hit) - 1 : 31;
            u.t = t0 + l;
            u.begin = u.s.before + u.head * u.s.head_len + done + __shfl_sync(0xffffffffu, incl - n, l);
            break;
        }
        done += __shfl_sync(0xffffffffu, incl, 31);
    }
    u.r = block_range(a, u.s.qlen, u.s.ctx, u.t);
    return u;
}

// Where the unit after u begins, or the line ends.
__device__ __forceinline__ long long unit_end(const Args& a, const Unit& u) {
    return u.begin + u.r.tiles + a.shape.unit_extra;
}

// The unit after u on the line (the caller knows that there is one).
template <typename Seqs>
__device__ __forceinline__ void next_unit(const Args& a, const Seqs& seqs, Unit& u) {
    u.begin = unit_end(a, u);
    if (++u.t >= token_blocks(a, u.s.qlen)) {
        u.t = 0;
        if (++u.head >= a.num_kv_heads) {
            u.head = 0;
            do {
                ++u.b;
                if (u.b >= a.batch) return;
                u.s = seqs.get(u.b);
            } while (u.s.qlen == 0);
        }
    }
    u.r = block_range(a, u.s.qlen, u.s.ctx, u.t);
}

// Checks sequence b's entries and adds up its units, by one thread (WARP = false) or a whole
// warp.  Entries that do not fit the call's extents give no work: the rows stay as they were.
template <bool WARP>
__device__ __forceinline__ Seq load_seq(const Args& a, int b, bool& good) {
    const int lane = WARP ? threadIdx.x & 31 : 0;
    const int r0 = a.cu[b], r1 = a.cu[b + 1], ctx = a.ctx[b];
    good = r0 >= 0 && r1 >= r0 && r1 <= a.rows && ctx >= 0 && ctx <= kMostKeys &&
           ctx <= (long long)a.max_pages * a.page_size;
    Seq s;
    s.row0 = r0;
    s.qlen = good ? r1 - r0 : 0;
    s.ctx = ctx;
    s.pad = 0;
    s.before = 0;
    long long n = 0;
    const int blocks = token_blocks(a, s.qlen);
    for (int t = lane; t < blocks; t += WARP ? 32 : 1)
        n += block_range(a, s.qlen, ctx, t).tiles + a.shape.unit_extra;
    if (WARP) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    }
    s.head_len = n;
    return s;
}

__device__ __forceinline__ Line make_line(const Args& a, long long total) {
    Line ln;
    ln.total = total;
    // at least min_tiles a CTA, unless the line is so short that CTAs would stay idle for it
    // (bf16, single tokens: one per CTA 10.3 and two 14.3 us for 2 tiles, 18.4 and 16.4 for 128)
    ln.per_part = max((total + a.shape.max_parts - 1) / a.shape.max_parts,
                      (long long)(total > 64 ? a.shape.min_tiles : 1));
    ln.parts = (int)((total + ln.per_part - 1) / ln.per_part);
    return ln;
}

// The line of at most 32 sequences, by a whole warp: sequence b in lane b.
__device__ __forceinline__ Line lane_line(const Args& a, LaneSeqs& seqs) {
    const int lane = threadIdx.x & 31;
    seqs.mine = Seq{0, 0, 0, 0, 0, 0};
    long long n = 0;
    if (lane < a.batch) {
        bool good;
        seqs.mine = load_seq<false>(a, lane, good);
        if (!good) tag_merge_inline(&a.ws->status, a.epoch, kStatusMismatch, false);
        n = seqs.mine.head_len * a.num_kv_heads;
    }
    long long incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
    }
    seqs.mine.before = incl - n;
    return make_line(a, __shfl_sync(0xffffffffu, incl, 31));
}

// The line as this CTA sees it, by every thread of a block of THREADS; ends with a block
// barrier.  Laid out here (a thread per sequence: the host saw to it that they suffice),
// every CTA writes the same values to a.seqs, and reads its own.  `scratch`: one word per
// warp of shared memory.
template <int THREADS>
__device__ __forceinline__ Line get_line(const Args& a, long long* scratch) {
    if (!a.line_inline) {
        Line ln = *a.line;
        __syncthreads();
        return ln;
    }
    const int b = threadIdx.x, warp = b >> 5, lane = b & 31;
    if (blockIdx.x == 0 && b == 0) a.ws->epoch = a.epoch;
    Seq s;
    long long n = 0;
    if (b < a.batch) {
        bool good;
        s = load_seq<false>(a, b, good);
        if (!good) tag_merge_inline(&a.ws->status, a.epoch, kStatusMismatch, false);
        n = s.head_len * a.num_kv_heads;
    }
    long long incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long before = incl - n, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    if (b < a.batch) {
        s.before = before;
        a.seqs[b] = s;
    }
    __syncthreads();
    return make_line(a, total);
}

// Where a CTA leaves its part of a split unit: two slots per CTA, one for the unit that has
// begun by the start of its stretch of the line and one for a unit that begins after it.
__device__ __forceinline__ long long part_slot(long long part, bool begins_stretch) {
    return 2 * part + (begins_stretch ? 0 : 1);
}

// The parts of a split unit: those of CTAs first .. last, in that order.
struct Split {
    int first, last;
    bool from_start;     // the unit begins where CTA first's stretch does
    __device__ __forceinline__ long long slot(int part) const {
        return part_slot(part, part > first || from_start);
    }
};

__device__ __forceinline__ Split split_of(const Unit& u, long long per) {
    Split s;
    s.first = (int)(u.begin / per);
    s.last = (int)((u.begin + u.r.tiles - 1) / per);
    s.from_start = u.begin == s.first * per;
    return s;
}

// The arrival counts of split units sit in words tagged for the call, so that they need no
// reset before it.  The tag spreads the call's number over 32 bits (an odd factor, so no two
// calls share one): what happens to be in fresh memory is small numbers more often than not.
// claim_arrivals: each CTA of a split unit, before its part is counted, gives the word of
// `share` this call's tag (and the count zero) unless another has; long before the part is
// done, so that counting it in is a single atomic.  False once a launch of this call has given
// up (a replay has its tag): its counts are then short of some parts, so nothing more is counted
// and nothing merged from parts that are not all in.
__device__ __forceinline__ unsigned long long arrival_tag(const Args& a) {
    return (unsigned long long)(a.epoch * 0x9E3779B1u ^ 0x5BD1E995u) << 32;
}
__device__ __forceinline__ bool claim_arrivals(const Args& a, const Split& sp, int share) {
    const unsigned long long status = *reinterpret_cast<volatile unsigned long long*>(&a.ws->status);
    unsigned long long* w = a.arrivals + (long long)sp.first * kArrivals + share;
    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(w);
    const unsigned long long tag = arrival_tag(a);
    while (old >> 32 != tag >> 32) {   // a retry finds another part's tag: one at most
        const unsigned long long seen = atomicCAS(w, old, tag);
        if (seen == old) break;
        old = seen;
    }
    return (unsigned int)(status >> 32) != a.epoch || !((unsigned int)status & (kStatusTimeout | kStatusBounds));
}

// Counts one more part in, by one thread after its warp's (or block's) threads have written
// it and fenced; true for the last, which puts the count back to zero for a replay.
__device__ __forceinline__ bool arrive_last(const Args& a, const Split& sp, int share) {
    unsigned long long* w = a.arrivals + (long long)sp.first * kArrivals + share;
    const unsigned int before = (unsigned int)atomicAdd(w, 1ull);
    if (before != (unsigned int)(sp.last - sp.first)) return false;
    *reinterpret_cast<volatile unsigned long long*>(w) = arrival_tag(a);
    __threadfence();
    return true;
}

// Launches a merging kernel so that its blocks start as the attention kernel's leave
// (programmatic dependent launch); they wait for all of it before they read.
template <typename Kernel>
inline cudaError_t launch_merge(Kernel kernel, dim3 grid, const Args& a, cudaStream_t stream) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_tc(const Args& a, cudaStream_t stream);   // bf16
Shape shape_tc();

}  // namespace attn

// Byte offsets of a call's workspace: status header, line, sequences, partial results.
namespace attn {
struct Layout {
    size_t line, seqs, arrivals, splits, part_lse, part_o, bytes;
};
}  // namespace attn

cudaError_t launch_paged_attention(const attn::Args& a, cudaStream_t stream);
attn::Shape paged_attention_shape(int dtype, int dim);
attn::Layout paged_attention_layout(int dtype, int dim, int batch);

}  // namespace gdn
