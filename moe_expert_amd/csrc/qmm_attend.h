// qmm_attend.h -- the attention kernels over the paged key-value cache, for gfx950: one pass over the keys and
// values with the running maximum and sum of a softmax, split over the cache's length, and the join of the parts.
//
// For a row (token, head) at position p: z_j = scale q . k_j over the positions j it sees, out = sum_j
// exp(z_j - m) v_j / sum_j exp(z_j - m).
//
// A wave takes 32 positions a step against 16 rows of queries that share a head of keys (RT = 2: 32 rows).
// Scores come transposed, S^T = K Q^T by v_mfma_f32_16x16x32_f16: lane (n = l % 16, g = l / 16) gets, of row n,
// the positions 4g .. 4g+3 of both 16-position halves.  That is the operand of O^T = V^T P^T as it stands when
// the contraction runs over positions in the order (g, half, 0..3), so no weight moves between lanes, and every
// statistic of a row belongs to its lane.
//
// What is rounded beside binary32's own: queries and weights, which enter the products in two binary16 parts, 2^-22 of the
// value in all but no finer than 2^-25 after a power of two that puts the row's largest near 2^14, 2^-39 of that.  One part
// alone would cost 2^-11, the error of a binary16 output; more parts, to keep 2^-22 of a weight far below the row's
// largest, half as many instructions again.  A block's integers are exact in binary16 (as (u - 128) 2^-10 of the biased
// byte u), its scale joins behind the products of the keys (one instruction a score and block) and before those of the values,
// into the weights: there each block of the head has a power of two of its own, or one block's large scales would push
// another's weights to where the second part ends (blocks 2^-13 apart, most of the weight on a position whose values are
// zero: 7 times the bound of the binary32 sums with one power for all, a hundredth of it so).
//
// Bounds.  Binary16: the cache's bytes (32 sequences of 8192 positions, 4 heads of 128: 98 us, 5.5 TB/s).  Block formats:
// the vector instructions of a step, some 450 for 32 positions of q8_0 and 650 of iq4_nl at 128 wide, most of them to unpack
// the bytes and to scale and cut the weights once a block (62 us, 4.6 TB/s; 59 us, 2.6 TB/s); the matrix units are
// busy an eighth of the time.  Few positions: one load after the other (arguments, lengths, pages, keys), 5 us until
// the first step, 1 us behind the last, and the join's launch.
#pragma once

#include <type_traits>

#include "qmm_kv.h"

namespace qmm {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kAtLds = 80 * 1024 - 512;  // bytes of LDS of a workgroup of which two share a CU
constexpr int kAtStep = 32;      // positions a step
// Sequences that a workgroup plans by itself; beyond, a launch of its own (q8_0, 128 of up to 250 positions, which are not
// split: 13.8 us, with the launch 18.4; of up to 1000: 33.0, 33.7; 256 of up to 250: 32.0, with it 30.2; of up to 1000:
// 52.2, 49.2).
constexpr int kAtInline = 128;

// What a workgroup leaves of a tile that goes on beyond it: the tile's pieces (0: none) and which of them, and its rows.
struct Piece {
    int count, mine, first, rows;  // first: of the sequence's new tokens;  rows: the tile's, and 64 times the tile
};

struct AttendArgs {
    const void* q;
    void* out;
    float* lse;
    float* parts;            // pieces: [slot][head][rows (m), rows (l), rows * dim]
    Piece* pieces;           // [slot], or null: no tile has more than one piece
    const int32_t* plan;     // of attend_plan_kernel, or null
    int64_t ldq, ldo;
    KvSide k, v;
    KvPlace p;
    int nheads, group, qtype, otype;  // group: heads of queries a head of keys
    float scale;                      // times log2(e) / 4, which is finite for every scale
    int window;                       // 0: none
    int target, one, least;           // workgroups a head of keys, of one for every CU;  steps that a tile counts for at least
    int shift;                        // a unit of the split is 2^shift steps: no line has more than 2^29 units
    int vec;                          // out: groups of four values are aligned
    uint32_t per_group, per_target;  // kv_per() of them
};

// The kernel's argument where it is needed: read again from its segment rather than kept in scalar registers, of which
// there are too few for all that a loop of steps does not need.
__device__ __forceinline__ const AttendArgs& launch_args() {
    auto p = (const __attribute__((address_space(4))) AttendArgs*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttendArgs*)p;
}

// ------------------------------------------------------------------ what a workgroup does

// Quotients by n > 0 of numbers in [0, 2^31), exact: the reciprocal is within 2^-44 of its value, and (v + 1/2) / n no
// nearer to a whole number than 1 / (2 n).
struct Per {
    double per;
    __device__ __forceinline__ explicit Per(int n) {
        const double r = (double)__builtin_amdgcn_rcpf((float)n);
        per = r * __builtin_fma(-(double)n, r, 2.0);
    }
    __device__ __forceinline__ int down(int v) const { return (int)(((double)v + 0.5) * per); }
    __device__ __forceinline__ int up(int v) const { return v > 0 ? down(v - 1) + 1 : 0; }
};

// Sequence s as the split sees it.
struct SeqWork {
    int first, n, len;  // its first new token, how many, its length
    int base, steps;    // first position of the walk (a multiple of 16), steps of 32 from there
    int tiles, seq;
};

__device__ __forceinline__ int lane_of(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ int wave_total(int v) { return lane_of(wave_scan(v), 63); }

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int s, int rows) {
    SeqWork w;
    w.seq = s;
    int end;
    kv_segment(a.p, s, w.first, end);
    w.n = end - w.first;
    w.len = max(a.p.lens[s], 0);
    const int last = (int)min((int64_t)w.len, (int64_t)a.p.max_pages * a.p.page_size);
    w.base = a.window > 0 && w.len - w.n >= a.window ? (w.len - w.n - a.window + 1) & ~15 : 0;
    w.steps = w.n > 0 && last > w.base ? (last - w.base + kAtStep - 1) / kAtStep : 0;
    w.tiles = (int)(((int64_t)w.n * a.group + rows - 1) / rows);
    return w;
}

__device__ __forceinline__ SeqWork lane_work(const AttendArgs& a, int s, int rows) {
    return s < a.p.nseq ? seq_work(a, s, rows) : SeqWork{0, 0, 0, 0, 0, 0, 0};
}

// How a call is split.  Every tile of rows, sequence by sequence, takes its steps' place on a line, at least `least` of
// them (about what a tile costs beside its steps), and each of the workgroups of a head takes the same length of it: the
// pieces of tiles that lie there.  A tile that goes on beyond its workgroup's length is joined from its pieces;
// since a workgroup has at most one piece of a tile that began before and one of a tile that goes on, two places a
// workgroup hold all pieces.
//
// Where the pieces of a length c, every tile cut by itself, are no more than the workgroups, and c is not much longer
// than the equal share of the steps, tiles take whole lengths: a workgroup has one piece then, and pays once for what
// it does beside its steps (kAtCost steps of its time, about: 33 of up to 4096 take 23.5 us, 64 34.3; with 3 28.7 and 38.5, with
// 40 the same; 40 x 4096 48.0, with 3 46.0).
//
// A length is a multiple of a step for each of four waves: one where the pieces then are no more than the CUs (1 x 1024
// q8_0: 10.9 us, with two 13.0), else two (16 x 4 tokens, 192 wide, a window of 1000: 21.5 us, with one 23.4).
//
// Where a table holds up to kAtShort steps and the tiles fill the CUs by themselves, or half as many, and there are no
// more tiles than workgroups, nothing is split, which saves the join's launch (64 x 512 q8_0: 14.9 us, split 18.4;
// 16 x 256: 9.6, 10.5; but 16 x 512, a quarter of the CUs: 13.6, split 11.4).
constexpr int kAtCost = 12;
constexpr int kAtWaves = 4;
constexpr int kAtShort = 18;

// Of two workgroups on a CU the one that came first is served first and ends first (32 x 8192 q8_0: after 38.7 us, the
// other after 48.3), so where lengths are long the workgroups take the line in pairs, one of the first half and one
// of the second, and the first of a pair takes kAtMore sixteenths of a length more (1 x 131071 iq4_nl 36.6 us, with 1 37.0, with
// 5 35.4; 64 x 4096 q8_0 63.2, 64.2, 62.5; others the same).  Long is kAtLong steps (32 of up to 6000, 16 rows, 256 wide iq4_nl:
// 25.7 us, from 8 on 32.2; 33 x 4096 q8_0 41.8, from 64 on 43.1; but 5 x 4096 17.6, from 8 on 16.5).
constexpr int kAtLong = 16, kAtMore = 3;
struct Split {
    int pair, first;  // units of two workgroups, and of the first of them
    int all;          // of the line
    int whole;        // units that a tile takes a multiple of, or 0
    bool paired;      // workgroups of the first and the second half in turn
    // The place on the line of a workgroup, counted along it, and which of them a unit belongs to.
    __device__ __forceinline__ int begin(int run) const { return (run >> 1) * pair + (run & 1 ? first : 0); }
    __device__ __forceinline__ int run_of(const Per& per, int unit) const {
        const int p = per.down(unit);
        return 2 * p + (unit - p * pair >= first ? 1 : 0);
    }
};

// Units of a tile that hold steps (one if there are none, for the zeros), and its units.
__device__ __forceinline__ int live_units(const AttendArgs& a, int steps) { return max(1, (steps + (1 << a.shift) - 1) >> a.shift); }
__device__ __forceinline__ int least_units(const AttendArgs& a) { return max(a.least >> a.shift, 1); }
__device__ __forceinline__ int line_units(const AttendArgs& a, int steps) { return max(live_units(a, steps), least_units(a)); }
__device__ __forceinline__ int tile_units(const AttendArgs& a, int steps, const Split& s) {
    const int live = live_units(a, steps);
    return s.whole ? Per(s.whole).up(live) * s.whole : max(live, least_units(a));
}

// units, tiles, tokens: of all sequences (line_units() of each tile); lengths(len): how many whole lengths all tiles
// take.  Offsets that decrease give more tokens than there are, of which units and tiles may not hold the count: nothing is
// done then.
template <class F>
__device__ __forceinline__ Split line_split(const AttendArgs& a, int units, int tiles, int64_t tokens, F lengths) {
    const bool many = tokens > a.p.ntok;
    if (!a.pieces && !a.plan)  // a workgroup a tile
        return Split{2 * kAtShort, kAtShort, many ? 0 : tiles * kAtShort, kAtShort, false};
    Split s;
    const int target = a.target, step = max(kAtWaves >> a.shift, 1);
    const auto rounded = [&](int len) { return max((len + step - 1) & -step, step); };  // as many steps for every wave
    uint32_t rest;
    const int share = (int)kv_divide(units, target, a.per_target, rest) + (rest ? 1 : 0);
    int even = rounded(share), count = lengths(even);
    if (even < 2 * step && count > a.one) {
        even = 2 * step;
        count = lengths(even);
    }
    if (count > a.one && count <= a.one + a.one / 8) {
        // rather a step more for all than two workgroups for a few CUs (32 of up to 6000, 16 rows, 256 wide iq4_nl: 25.7 us, without
        // 28.3; up to a third more of them: the same, but 5 x 4096 q8_0 16.1, an eighth 17.6)
        even += step;
        count = lengths(even);
    }
    int len = even;
    bool whole = true;
    s.paired = even >= kAtLong >> a.shift && target > a.one;
    const int pairs = s.paired ? lengths(2 * even) : 0;
    if (s.paired && 2 * pairs <= target) {
        count = pairs;
        s.whole = 2 * even;
    } else {
        if (count > target && target > tiles / 2) {
            // not the equal share, but one that leaves half a length a tile
            const int left = target - tiles / 2;
            len = rounded(Per(left).up(units));
            count = len > even + (kAtCost >> a.shift) ? count : lengths(len);
        }
        whole = count <= target;
        if (!whole) len = max(share, least_units(a));
        s.paired = s.paired && !whole;
        s.whole = whole ? len : 0;
    }
    s.pair = 2 * len;
    s.first = s.paired ? len + ((len * kAtMore / 16 + step - 1) & -step) : len;
    s.all = many ? 0 : whole ? count * s.whole : units;
    if (many) s.pair = s.first = 0;  // (nobody's place is below 0)
    return s;
}

// A tile on the line: its first unit.
struct Tile {
    SeqWork w;
    int tile, at, live, units;
};

// The split, by every wave for itself; w: the lane's sequence of the first 64, for find_tile.
__device__ __forceinline__ Split find_split(const AttendArgs& a, int rows, SeqWork& w) {
    const int lane = threadIdx.x & 63, nseq = a.p.nseq;
    if (a.plan) return Split{a.plan[0], a.plan[1], a.plan[2], 0, a.plan[1] * 2 != a.plan[0]};
    int units = 0, tokens = 0, tiles = 0;
    for (int j = (nseq - 1) & ~63; j >= 0; j -= 64) {
        w = lane_work(a, j + lane, rows);
        units += wave_total(w.tiles * line_units(a, w.steps));
        tokens += wave_total(w.n);
        tiles += wave_total(w.tiles);
    }
    return line_split(a, units, tiles, tokens, [&](int len) {
        int all = 0;
        const Per per(len);
        for (int j = 0; j < nseq; j += 64) {
            const SeqWork v = j ? lane_work(a, j + lane, rows) : w;
            all += wave_total(v.tiles * per.up(live_units(a, v.steps)));
        }
        return all;
    });
}

// The tile that unit `at` of the line belongs to; w: the lane's sequence of the first 64.
__device__ __forceinline__ Tile find_tile(const AttendArgs& a, const Split& s, int at, int rows, const SeqWork& first) {
    const int lane = threadIdx.x & 63, nseq = a.p.nseq;
    Tile t;
    int before = 0;
    if (a.plan) {
        const int32_t* units = a.plan + 3;  // before each sequence, and all
        const int stride = (nseq + 63) / 64;
        int seq = stride * __popcll(__ballot(units[min((lane + 1) * stride, nseq)] <= at));
        const int end = min(seq + stride, nseq);
        int more = 0;
        for (int j = seq; j < end; j += 64) more += __popcll(__ballot(j + lane < end && units[min(j + lane + 1, nseq)] <= at));
        seq = __builtin_amdgcn_readfirstlane(seq + more);
        t.w = seq_work(a, seq, rows);
        before = units[seq];
    } else {
        for (int j = 0; j < nseq; j += 64) {
            const SeqWork w = j ? lane_work(a, j + lane, rows) : first;
            const int mine = w.tiles * tile_units(a, w.steps, s), upto = wave_scan(mine), total = lane_of(upto, 63);
            if (at < before + total) {
                const int l = __popcll(__ballot(before + upto <= at));
                t.w.first = lane_of(w.first, l);
                t.w.n = lane_of(w.n, l);
                t.w.len = lane_of(w.len, l);
                t.w.base = lane_of(w.base, l);
                t.w.steps = lane_of(w.steps, l);
                t.w.tiles = lane_of(w.tiles, l);
                t.w.seq = j + l;
                before += lane_of(upto - mine, l);
                break;
            }
            before += total;
        }
    }
    t.live = live_units(a, t.w.steps);
    t.units = tile_units(a, t.w.steps, s);
    t.tile = t.w.tiles > 1 ? Per(t.units).down(at - before) : 0;
    t.at = before + t.tile * t.units;
    return t;
}

// ------------------------------------------------------------------ values as the matrix instructions take them

template <int TYPE, int NB>
struct Side {
    static constexpr int kFactor = TYPE == kKvF16 ? 64 * NB : TYPE == kKvQ8 ? 32 * NB : 16 * NB;  // bytes of a position
    static constexpr int kScale = TYPE == kKvF16 ? 0 : 2 * NB;
    static constexpr int kRow = kFactor + kScale;
};

// ------------------------------------------------------------------ blocks on their way through LDS

// Lane l's 16 bytes at base + offset + IMM to lds + IMM + 16 l (lds and base are the wave's).  Not the builtin: behind that
// the compiler waits for every load on its way before any read of LDS.  Its own counts stay safe: it waits for more
// than it means to.  (m0 is no register that it keeps anything in.)
// (Five states from base's last v_readlane to its use.)  The first LANES lanes of a wave of 64 whose lanes are all
// active.
template <int IMM, int LANES>
__device__ __forceinline__ void to_lds(char* lds, const char* base, uint32_t offset) {
    static_assert(IMM >= 0 && IMM < 4096 && LANES > 0 && LANES <= 64, "the instruction's offset, a wave");
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    if constexpr (LANES == 64) {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3" : : "s"(at), "v"(offset), "s"(base), "n"(IMM) : "memory");
    } else {
        constexpr uint32_t kLow = LANES >= 32 ? ~0u : (1u << (LANES & 31)) - 1, kHigh = LANES > 32 ? (1u << ((LANES - 32) & 31)) - 1 : 0;
        asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %4\n\ts_mov_b32 exec_hi, %5\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3\n\t"
                     "s_mov_b64 exec, -1"
                     : : "s"(at), "v"(offset), "s"(base), "n"(IMM), "n"(kLow), "n"(kHigh) : "memory");
    }
}

// Orders LDS accesses of the lanes of a wave, which run in step.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Bits 15 and 31: whether each of two halves is not finite.  (Many of them are joined without a compare each.)
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) { return ((v & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }
// The halves that are finite, zeros for the others.
__device__ __forceinline__ uint32_t finite_halves(uint32_t v) { return v & ~((odd_halves(v) >> 15) * 0xFFFFu); }

template <int CTRL>
__device__ __forceinline__ u16x2 dpp_pair(u16x2 v) { return __builtin_bit_cast(u16x2, dpp_i<CTRL>(__builtin_bit_cast(int, v))); }
// The least of the 16 lanes of a row, both halves apart; the most of the lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ u16x2 min16_pair(u16x2 v) {
    v = __builtin_elementwise_min(v, dpp_pair<0xB1>(v));
    v = __builtin_elementwise_min(v, dpp_pair<0x4E>(v));
    v = __builtin_elementwise_min(v, dpp_pair<0x141>(v));
    return __builtin_elementwise_min(v, dpp_pair<0x140>(v));
}
__device__ __forceinline__ u16x2 rows_max16(u16x2 v) {
    const int x = __builtin_bit_cast(int, v);
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_elementwise_max(__builtin_bit_cast(u16x2, (int)r[0]), __builtin_bit_cast(u16x2, (int)r[1]));
    const int y = __builtin_bit_cast(int, v);
    r = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __builtin_elementwise_max(__builtin_bit_cast(u16x2, (int)r[0]), __builtin_bit_cast(u16x2, (int)r[1]));
}

// 32 positions of a block format, as they lie in a page: the factors of both 16-position halves, then their scales,
// copied by the wave itself 16 bytes a lane without passing registers, so that whole steps are on their way
// while one is worked on.  A piece of 16 bytes keeps its row and goes, where a row is a power of two of them, to
// place c ^ turn(row): sixteen lanes that read the same piece of as many rows meet different banks.
template <int TYPE, int NB>
struct Stage {
    static constexpr int kFactor = Side<TYPE, NB>::kFactor, kRowPieces = kFactor / 16;
    static constexpr int kHalf = kFactor;  // pieces of 16 rows
    static constexpr int kHalfLoads = (kHalf + 63) / 64, kLoads = 2 * (kHalfLoads + 1);
    static constexpr int kScales = 32 * kHalf;  // their place
    static constexpr int kBytes = kScales + 64 * NB;
    static constexpr bool kTurn = (kRowPieces & (kRowPieces - 1)) == 0;
    // Loads of a lane whose offsets differ by more than the instruction's: 64 pieces on, the turn of the row is the
    // same but for rows of 16 pieces.
    static constexpr int kOffsets = kRowPieces == 16 ? 2 : 1;

    __device__ static __forceinline__ int turn(int row) {
        return !kTurn ? 0 : kRowPieces >= 8 ? row & 7 : row / (8 / kRowPieces) & (kRowPieces - 1);
    }
    // Where byte `at` of row `row` (of 32) lies.
    __device__ static __forceinline__ int place(int row, int at) { return (row * kRowPieces + (at / 16 ^ turn(row))) * 16 + at % 16; }

    uint32_t offset[kOffsets];
    __device__ __forceinline__ Stage(int lane) {
#pragma unroll
        for (int i = 0; i < kOffsets; ++i) {
            const int p = 64 * i + lane, row = p / kRowPieces;
            offset[i] = row * kFactor + 16 * (p % kRowPieces ^ turn(row));
        }
    }
    // One half: 16 positions, whose factors begin at rows and whose scales are `scales` bytes on.
    __device__ __forceinline__ void fetch(int lane, char* lds, int h, const char* rows, int scales) const {
        fetch_rows<0>(lds + 16 * kHalf * h, rows);
        to_lds<0, 2 * NB>(lds + kScales + 32 * NB * h, rows + scales, 16 * lane);
    }
    template <int I>
    __device__ __forceinline__ void fetch_rows(char* lds, const char* rows) const {
        if constexpr (I < kHalfLoads) {
            constexpr int kBase = I % kOffsets, kImm = 1024 * (I - kBase);
            to_lds<kImm, kHalf >= 64 * I + 64 ? 64 : kHalf - 64 * I>(lds + 1024 * kBase, rows, offset[kBase]);
            fetch_rows<I + 1>(lds, rows);
        }
    }
    // N bytes of a row from `at` on; N divides 16 or is a multiple of it where rows are turned.
    template <int N>
    __device__ static __forceinline__ void read(uint32_t* w, const char* lds, int row, int at) {
        if constexpr (!kTurn && (N == 3 || N == 6 || N == 12)) {
            // The dwords around them, one by one: the compiler would join them to reads of 8 bytes, which take four times as long
            // from addresses that are no multiples of 8 (32 sequences of 4096, 96 wide, iq4_nl: 44 us, apart 36).
            constexpr int kDwords = N == 12 ? 3 : 2;
            const auto p = (const volatile __attribute__((address_space(3))) uint32_t*)(const __attribute__((address_space(3))) char*)(lds + row * kFactor + (at & ~3));
            uint32_t some[kDwords];
#pragma unroll
            for (int i = 0; i < kDwords; ++i) some[i] = p[i];
            if constexpr (N == 12) {
#pragma unroll
                for (int i = 0; i < 3; ++i) w[i] = some[i];
            } else {
                w[0] = align8(some[1], some[0], at);
                if constexpr (N == 6) w[1] = some[1] >> (8 * (at & 3)) & 0xFFFFu;
            }
        } else if constexpr (!kTurn) {
            if constexpr (N % 4) w[N / 4] = 0;
            constexpr int kAlign = N % 16 == 0 ? 16 : N % 8 == 0 ? 8 : N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
            __builtin_memcpy(w, __builtin_assume_aligned(lds + row * kFactor + at, kAlign), N);
        } else if constexpr (N >= 16) {
#pragma unroll
            for (int i = 0; i < N / 16; ++i) __builtin_memcpy(w + 4 * i, __builtin_assume_aligned(lds + place(row, at + 16 * i), 16), 16);
        } else {
            if constexpr (N % 4) w[N / 4] = 0;
            __builtin_memcpy(w, __builtin_assume_aligned(lds + place(row, at), N), N);
        }
    }
    // The scales of positions 4g .. 4g+3 of a half.
    __device__ static __forceinline__ void scales(uint32_t* d, const char* lds, int h, int g) {
        __builtin_memcpy(d, __builtin_assume_aligned(lds + kScales + (32 * h + 8 * g) * NB, 8), 8 * NB);
    }
    // Of the 4 NB dwords of scales of positions 4g .. 4g+3 of both halves the magnitudes of the ones that a lane's place n among
    // 16 falls to, each of two blocks; and whether one of them has binary16 bits of more than `most`.
    static constexpr int kParts = (4 * NB + 15) / 16;
    __device__ static __forceinline__ int part(int n, int i) { return min(n + 16 * i, 4 * NB - 1); }
    __device__ static __forceinline__ void parts(const char* lds, int n, int g, u16x2 (&v)[kParts]) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int j = part(n, i);
            v[i] = __builtin_bit_cast(u16x2, *(const uint32_t*)(lds + kScales + (32 * (j / (2 * NB)) + 8 * g) * NB + 4 * (j % (2 * NB))) & 0x7FFF7FFFu);
        }
    }
    __device__ static __forceinline__ bool above(const u16x2 (&v)[kParts], const u16x2 (&most)[kParts]) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            any |= __builtin_bit_cast(uint32_t, __builtin_elementwise_max(v[i], most[i])) != __builtin_bit_cast(uint32_t, most[i]);
        return any;
    }
    // The step's scales without those that are not finite, by the whole wave.
    __device__ static __forceinline__ void keep_finite(char* lds, int lane) {
        uint32_t* w = (uint32_t*)(lds + kScales);
        for (int i = lane; i < 16 * NB; i += 64) w[i] = finite_halves(w[i]);
        wave_fence();
    }
    // The blocks' largest of a step, from all lanes' parts: of two, four or eight blocks the lanes whose n are the same modulo
    // their pairs hold the same blocks.
    static constexpr bool kWhole = (NB & (NB - 1)) == 0;
    __device__ static __forceinline__ void largest(const u16x2 (&v)[kParts], u16x2 (&most)[(NB + 1) / 2]) {
        static_assert(kWhole, "pairs of blocks that divide the lanes of a quad");
        u16x2 w = v[0];
#pragma unroll
        for (int i = 1; i < kParts; ++i) w = __builtin_elementwise_max(w, v[i]);
        if constexpr (NB < 4) w = __builtin_elementwise_max(w, dpp_pair<0xB1>(w));
        if constexpr (NB < 8) w = __builtin_elementwise_max(w, dpp_pair<0x4E>(w));
        w = __builtin_elementwise_max(w, dpp_pair<0x124>(w));  // row_ror 4, 8
        w = __builtin_elementwise_max(w, dpp_pair<0x128>(w));
        w = rows_max16(w);
        most[0] = dpp_pair<0x00>(w);
        if constexpr (NB >= 4) most[1] = dpp_pair<0x55>(w);
        if constexpr (NB >= 8) {
            most[2] = dpp_pair<0xAA>(w);
            most[3] = dpp_pair<0xFF>(w);
        }
    }
    // What is compared there, of the values for blocks 2i and 2i + 1 in v[i].
    __device__ static __forceinline__ void share(int n, const u16x2 (&v)[(NB + 1) / 2], u16x2 (&most)[kParts]) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int first = 2 * part(n, i) % NB;  // of the blocks
            if constexpr (NB % 2 == 0) {
                most[i] = v[0];
#pragma unroll
                for (int b = 1; b < NB / 2; ++b) most[i] = first == 2 * b ? v[b] : most[i];
            } else {
                static_assert(NB % 2 == 0 || NB == 3, "blocks (0, 1), (2, 0), (1, 2)");
                most[i] = first == 0 ? v[0] : first == 2 ? u16x2{v[1].x, v[0].x} : u16x2{v[0].y, v[1].x};
            }
        }
    }
};

// At most n vector memory operations of the wave outstanding; what is read from LDS afterwards is what the others
// brought there.
template <int N>
__device__ __forceinline__ void arrived() {
    static_assert(N < 64, "six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0F70);
    asm volatile("" ::: "memory");
}
// What this wave reads from LDS is in its registers, so the place may be written.
__device__ __forceinline__ void taken() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}

// ------------------------------------------------------------------ operands

// Two biased bytes u = q + 128, which perm laid into the low bytes of two halves, are u 2^-24 as binary16 values: to
// q 2^-10.  (They could enter the products as they are, and what 128 in their place gives be taken from the sums.  That
// is no faster, the matrix instructions wait for the others, and costs digits: 128 times a long context's weights is
// far above the sum of its values.  8 sequences of 4096 positions, q8_0, were 9e-6 off so, and are 2e-7.)
__device__ __forceinline__ uint32_t byte_pair(uint32_t x) {
    const half2_t scale = {(_Float16)16384.0f, (_Float16)16384.0f}, bias = {(_Float16)-0.125f, (_Float16)-0.125f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, x), scale, bias));
}
constexpr uint32_t pair_sel(int low, int high) { return 0x0C000C00u | (uint32_t)low | (uint32_t)high << 16; }

// Biased levels of a dword of index bytes, the low halves' and the high halves'.
__device__ __forceinline__ void levels(uint32_t q, uint32_t& lo, uint32_t& hi) {
    lo = iq4nl_lookup_u(q & 0x07070707u, ((q >> 1) & 0x04040404u) | 0x03020100u);
    hi = iq4nl_lookup_u((q >> 4) & 0x07070707u, ((q >> 5) & 0x04040404u) | 0x03020100u);
}

__device__ __forceinline__ half8_t as_half8(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return __builtin_bit_cast(half8_t, u32x4{x, y, z, w}); }

// The keys of 16 positions: lane (position n, quarter g) holds of every block b the eight dims 32b + 16i + 4g +
// (0..3), i = 0, 1 (binary16: 32b + 8g + (0..7)).
template <int TYPE, int NB>
struct Keys {
    static constexpr int kBytes = TYPE == kKvF16 ? 0 : Side<TYPE, NB>::kFactor / 4;
    uint32_t w[TYPE == kKvF16 ? 4 * NB : kBytes / 4];
    uint32_t d[TYPE == kKvF16 ? 1 : 2 * NB];  // scales [position 4g + r][block], two a dword

    // Of binary16, from memory; block formats come through LDS.
    __device__ __forceinline__ void load(int lane, const char* rows) {
        static_assert(TYPE == kKvF16, "block formats are staged");
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            u32x4 v;
            load_block(v, lane, rows, b);
            __builtin_memcpy(w + 4 * b, &v, 16);
        }
    }
    __device__ static __forceinline__ void load_block(u32x4& v, int lane, const char* rows, int b) {
        const char* p = rows + (uint32_t)((lane & 15) * (64 * NB) + 16 * (lane >> 4));
        __builtin_memcpy(&v, __builtin_assume_aligned(p + 64 * b, 16), 16);
    }
    __device__ __forceinline__ void read(int lane, int h, const char* lds) {
        const int n = lane & 15, g = lane >> 4;
        Stage<TYPE, NB>::template read<kBytes>(w, lds, 16 * h + n, g * kBytes);
        Stage<TYPE, NB>::scales(d, lds, h, g);
    }
    // Biases the bytes of q8_0, looks the levels of iq4_nl up.
    struct Ready {
        uint32_t a[TYPE == kKvF16 ? 4 * NB : kBytes / 4], b[TYPE == kKvIq4 ? kBytes / 4 : 1];
    };
    __device__ __forceinline__ void ready(Ready& r) const {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(w) / 4); ++i) {
            if constexpr (TYPE == kKvF16) r.a[i] = w[i];
            else if constexpr (TYPE == kKvQ8) r.a[i] = w[i] ^ 0x80808080u;
            else levels(w[i], r.a[i], r.b[i]);
        }
    }
    __device__ static __forceinline__ half8_t block(const Ready& r, int b) {
        if constexpr (TYPE == kKvF16) return as_half8(r.a[4 * b], r.a[4 * b + 1], r.a[4 * b + 2], r.a[4 * b + 3]);
        uint32_t x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (TYPE == kKvQ8) {
                const int at = (m * NB + b) * 2;
                x[m] = byte_pair(perm(r.a[at / 4], r.a[at / 4], pair_sel(at % 4, at % 4 + 1)));
            } else {
                const int at = m * NB + b;
                x[m] = byte_pair(perm(r.b[at / 4], r.a[at / 4], pair_sel(at % 4, at % 4 + 4)));
            }
        }
        return as_half8(x[0], x[1], x[2], x[3]);
    }
    __device__ __forceinline__ float scale(int r, int b) const {
        const int i = r * NB + b;
        return (float)__builtin_bit_cast(half2_t, d[i / 2])[i & 1];
    }
};

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7C00u) == 0x7C00u; }

// The values of 32 positions: lane (n, g) holds, of the positions 4g .. 4g+3 of both halves, the dims that
// row n of the 2 NB operands V^T takes: tile (b, i) dim 32b + 16i + n (binary16: tile j dim 2 NB n + j).
template <int TYPE, int NB>
struct Values {
    static constexpr int kBytes = Side<TYPE, NB>::kFactor / 16;
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[8][kWords];
    uint32_t d[2][TYPE == kKvF16 ? 1 : 2 * NB];  // scales [half][position 4g + r][block]

    __device__ __forceinline__ void load(int lane, int half, const char* rows) {
        static_assert(TYPE == kKvF16, "block formats are staged");
        const char* p = rows + (uint32_t)(4 * (lane >> 4) * Side<TYPE, NB>::kFactor + (lane & 15) * kBytes);
#pragma unroll
        for (int r = 0; r < 4; ++r) __builtin_memcpy(w[4 * half + r], p + r * Side<TYPE, NB>::kFactor, kBytes);
    }
    __device__ __forceinline__ void read(int lane, const char* lds) {
        const int n = lane & 15, g = lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int r = 0; r < 4; ++r) Stage<TYPE, NB>::template read<kBytes>(w[4 * h + r], lds, 16 * h + 4 * g + r, n * kBytes);
        }
        read_scales(lane, lds);
    }
    __device__ __forceinline__ void read_scales(int lane, const char* lds) {
#pragma unroll
        for (int h = 0; h < 2; ++h) Stage<TYPE, NB>::scales(d[h], lds, h, lane >> 4);
    }
    __device__ __forceinline__ _Float16 scale(int x, int b) const {
        const int i = (x & 3) * NB + b;
        return __builtin_bit_cast(half2_t, d[x >> 2][i / 2])[i & 1];
    }
    // The binary16 bits of the largest magnitude among each block's scales, of all positions or of those seen, blocks 2i and
    // 2i + 1 in most[i]; by all lanes of a row.
    static constexpr int kPairs = (NB + 1) / 2;
    template <bool MASKED>
    __device__ __forceinline__ void largest(int seen, u16x2 (&most)[kPairs]) const {
        constexpr int kTurn = NB % 2 ? NB : NB / 2;  // dwords until their two blocks are the same again
        u16x2 of[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) of[i] = u16x2{0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                uint32_t v = d[h][i] & 0x7FFF7FFFu;
                if constexpr (MASKED) {
                    const int x = 4 * h + 2 * i / NB, y = 4 * h + (2 * i + 1) / NB;
                    const uint32_t a = (uint32_t)((int)((uint32_t)seen << (31 - x)) >> 31), b = (uint32_t)((int)((uint32_t)seen << (31 - y)) >> 31);
                    v &= x == y ? a : (a & 0xFFFFu) | (b & 0xFFFF0000u);
                }
                of[i % kTurn] = __builtin_elementwise_max(of[i % kTurn], __builtin_bit_cast(u16x2, v));
            }
        if constexpr (NB % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) most[i] = of[i];
        } else {
            static_assert(NB % 2 == 0 || NB == 3, "blocks (0, 1), (2, 0), (1, 2)");
            most[0] = __builtin_elementwise_max(of[0], u16x2{of[1].y, of[2].x});
            most[1] = u16x2{of[1].x > of[2].y ? of[1].x : of[2].y, 0};
        }
#pragma unroll
        for (u16x2& v : most) v = rows_max16(v);
    }
    // Whether a binary16 value is not finite: its product with zero is a NaN then, one instruction a dword.
    __device__ __forceinline__ bool any_odd() const {
        const half2_t zero = {0, 0};
        half2_t sum[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int i = 0; i < kWords; ++i) sum[x & 3] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, w[x][i]), zero, sum[x & 3]);
        return odd_halves(__builtin_bit_cast(uint32_t, (sum[0] + sum[1]) + (sum[2] + sum[3]))) != 0;
    }
    // The scales as they are loaded, two a register, also past a branch that may change them.
    __device__ __forceinline__ void keep_words() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) asm("" : "+v"(d[h][i]));
    }
    // Biased bytes; of iq4_nl the levels, where two half dwords of neighbouring positions share a lookup.
    struct Ready {
        uint32_t a[8][kWords], b[TYPE == kKvIq4 ? 8 : 1][kWords];
    };
    __device__ __forceinline__ void ready(Ready& r) const {
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (TYPE == kKvF16) r.a[x][i] = w[x][i];
                else if constexpr (TYPE == kKvQ8) r.a[x][i] = w[x][i] ^ 0x80808080u;
                else if (kBytes % 4 != 2 || i < kWords - 1) levels(w[x][i], r.a[x][i], r.b[x][i]);
                else if (x & 1) {
                    levels(w[x - 1][i] | w[x][i] << 16, r.a[x - 1][i], r.b[x - 1][i]);
                    r.a[x][i] = r.a[x - 1][i];
                    r.b[x][i] = r.b[x - 1][i];
                }
            }
    }
    __device__ static __forceinline__ half8_t tile(const Ready& r, int t) {
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (TYPE == kKvF16) {
                o[m] = perm(r.a[2 * m + 1][t / 2], r.a[2 * m][t / 2], t & 1 ? 0x07060302u : 0x05040100u);
            } else if constexpr (TYPE == kKvQ8) {
                o[m] = byte_pair(perm(r.a[2 * m + 1][t / 4], r.a[2 * m][t / 4], pair_sel(t % 4, t % 4 + 4)));
            } else {
                const int b = t / 2, i = b / 4, shared = kBytes % 4 == 2 && i == kWords - 1 ? 2 : 0;
                const uint32_t lo = t & 1 ? r.b[2 * m][i] : r.a[2 * m][i], hi = t & 1 ? r.b[2 * m + 1][i] : r.a[2 * m + 1][i];
                o[m] = byte_pair(perm(hi, lo, pair_sel(b % 4, b % 4 + 4 + shared)));
            }
        }
        return as_half8(o[0], o[1], o[2], o[3]);
    }
    // The dim of row m of tile t.
    __device__ static __forceinline__ int dim(int t, int m) { return TYPE == kKvF16 ? 2 * NB * m + t : 16 * t + m; }
};

// Constants that the compiler does not see through: a product and sum with them stays one v_fma_mix_f32, which
// takes binary16 factors as they are; a plain difference or product would convert them first.
struct Mix {
    float minus, zero;
    __device__ __forceinline__ Mix() : minus(-1.0f), zero(0.0f) { asm("" : "+s"(minus), "+s"(zero)); }
    __device__ __forceinline__ float rest(float x, _Float16 h) const { return __builtin_fmaf((float)h, minus, x); }
    __device__ __forceinline__ float product(float x, _Float16 h) const { return __builtin_fmaf((float)h, x, zero); }
    __device__ __forceinline__ float product_rest(float x, _Float16 h, _Float16 near) const { return __builtin_fmaf((float)h, x, -(float)near); }
};

// Two binary16 parts of pairs of values: the nearest, and the nearest of what is left.
__device__ __forceinline__ void two_parts(const Mix& mix, float x, float y, uint32_t& hi, uint32_t& lo) {
    const half2_t h = __builtin_convertvector((float2_t{x, y}), half2_t);
    const float2_t rest = {mix.rest(x, h.x), mix.rest(y, h.y)};
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, half2_t));
}

// The same of eight values' products with factors.  (All pairs' nearest before what they leave: a conversion waits for the two
// values that it takes.  v_fma_mixlo_f16 and v_fma_mixhi_f16 would take four instructions a pair, these are six, but
// take longer: 1 x 131071 q8_0/iq4_nl 34.3 us, these 33.1.)
template <class F>
__device__ __forceinline__ void scaled_parts(const Mix& mix, const float (&u)[8], F factor, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2_t p = {mix.product(u[2 * i], factor(2 * i)), mix.product(u[2 * i + 1], factor(2 * i + 1))};
        hi[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, half2_t));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const half2_t h = __builtin_bit_cast(half2_t, hi[i]);
        const float2_t rest = {mix.product_rest(u[2 * i], factor(2 * i), h.x), mix.product_rest(u[2 * i + 1], factor(2 * i + 1), h.y)};
        lo[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, half2_t));
    }
}

// Maximum and sum over the lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ float rows_max(float v) {
    const int x = __builtin_bit_cast(int, v);
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_fmaxf(__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1]));
    const int y = __builtin_bit_cast(int, v);
    r = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
    const int x = __builtin_bit_cast(int, v);
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
    const int y = __builtin_bit_cast(int, v);
    r = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
}

// A row's fold of a block of values, a power of two: its weights times the block's scales times the fold are what is cut into
// binary16 parts.  The largest scale that the row has seen of the block has a product in [2^13, 2^15) with it.  2^e / fold:
constexpr uint32_t kFoldMost = (127u + 38u) << 23;  // (the least scale is 2^-24)
template <int E>
__device__ __forceinline__ float over(uint32_t fold) {
    return __builtin_bit_cast(float, ((127u + E + 127u) << 23) - fold);
}

__device__ __forceinline__ void store4(const float* v, void* p, int64_t i, int type, int vec) {
    if (vec && type == kF32) {
        *(float4_t*)((float*)p + i) = float4_t{v[0], v[1], v[2], v[3]};
    } else if (vec) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = type == kBin16 ? f2h(v[e]) : f2bf(v[e]);
        *(u32x2*)((uint16_t*)p + i) = u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_value(p, i + e, type, v[e]);
    }
}

// Four dims of row r (of its sequence's) of a head of keys, and with the first of them the row's lse.
__device__ __forceinline__ void write_row(const AttendArgs& a, int first, int head, int r, int d, float4_t f, float most, float sum) {
    uint32_t rest;
    const int token = (int)kv_divide(r, a.group, a.per_group, rest), h = head * a.group + (int)rest;
    const float v[4] = {f[0], f[1], f[2], f[3]};
    store4(v, a.out, (first + token) * a.ldo + (int64_t)h * a.p.dim + d, a.otype, a.vec);
    if (d == 0 && a.lse)
        a.lse[(int64_t)(first + token) * a.nheads + h] = sum != 0.0f ? most * 0.693147180559945f + __logf(sum) : -INFINITY;
}

// The weight of a result whose maximum is m beside one of a maximum `top`.  At m = -inf its sums are zeros, or NaN.
__device__ __forceinline__ float beside(float m, float top) { return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top); }

// Floats of a slot and head.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// ------------------------------------------------------------------ the pass

struct Nothing {
    __device__ Nothing(int) {}
};

// How a pair of formats, a width and a number of row tiles are run: waves of a workgroup, whether keys and values pass
// through LDS on their way (block formats do), and how many steps ahead they set out.  Binary16 keys are read into
// registers, a step ahead: before the weights, or after the values where the registers do not hold both (32 x 4096, 192
// wide, values of q8_0: 67 us, before the weights 89).
template <int KT, int VT, int NB, int RT>
struct Shape {
    static constexpr bool kStaged = KT != kKvF16;
    static constexpr int kKeys = kStaged ? Stage<KT, NB>::kBytes : 0, kVals = VT != kKvF16 ? Stage<VT, NB>::kBytes : 0;
    static constexpr int kQueries = RT * NB * 2 * 64 * 16;
    static constexpr int kWaves = kQueries + 4 * (kKeys + kVals) > kAtLds ? 8 : 4;
    static constexpr bool kTwo = kWaves == 4 && kQueries + 8 * (kKeys + kVals) <= kAtLds;
    static constexpr bool kEarly = !kStaged && (VT == kKvF16 ? NB < 8 : NB * RT <= 4) && kTwo;
    static constexpr int kDepth = kTwo && (kStaged || kEarly) ? 2 : 1;
    static constexpr int kRing = kDepth * (kKeys + kVals);  // bytes a wave
    static constexpr int kRows = 16 * RT, kPitch = 32 * NB + 4;
    static constexpr int kSums = kWaves * kRows * (kPitch + 2) * 4;  // of the waves, at the end, in place of all else
    static constexpr int kOdd = KT == kKvF16 && VT == kKvF16 ? kRows * kAtStep * 4 + 64 * NB : 0;  // bytes a wave: values that are not finite
    static constexpr int kLoop = kQueries + kWaves * (kRing > kOdd ? kRing : kOdd);
    static constexpr int kBytes = kLoop > kSums ? kLoop : kSums;
};

// The queries' parts lie in LDS, read again each step (two 16-byte reads a block), which leaves the registers to the keys
// and values.
// A piece of a tile: `count` steps of it from step `from` on.  slot: its place, or -1 for a whole tile.
template <int KT, int VT, int NB, int RT>
__device__ __forceinline__ void attend_piece(const SeqWork& w, int tile, int from, int count, char* lds, float* lc,
                                             int head, int slot) {
    const AttendArgs& a = launch_args();
    using S = Shape<KT, VT, NB, RT>;
    constexpr int kRows = 16 * RT, kDim = 32 * NB, kTiles = 2 * NB, kWaves = S::kWaves, kDepth = S::kDepth;
    constexpr bool kKeyBlocks = KT != kKvF16, kValBlocks = VT != kKvF16, kStaged = S::kStaged;
    constexpr bool kEarly = S::kEarly;
    // Queries, then what is on its way, wave by wave; at the end the sums of the waves in their place.
    auto& lq = *(uint32_t(*)[RT][NB][2][64][4])lds;
    auto& so = *(float(*)[kWaves][kRows][S::kPitch])lds;
    auto& lm = *(float(*)[kWaves][kRows])(lds + sizeof(so));
    auto& ll = *(float(*)[kWaves][kRows])(lds + sizeof(so) + sizeof(lm));
    static_assert(sizeof(so) + sizeof(lm) + sizeof(ll) == S::kSums, "the sums' place");
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // what depends on it is not kept from one piece to the next
    const int lane = tid & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // The rows of the tile: lane n's, the positions [rlo, rhi) that they see, and the same over all of them.
    const int row0 = tile * kRows, rows = min(kRows, w.n * a.group - row0), cap = a.p.max_pages * a.p.page_size;
    const auto token_of = [&](int r) {
        uint32_t rest;
        return (int)kv_divide(r, a.group, a.per_group, rest);
    };
    const auto low = [&](int pos) { return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0; };
    const int pos0 = w.len - w.n + token_of(row0), pos1 = w.len - w.n + token_of(row0 + rows - 1);
    const int lo_min = low(pos0), lo_max = low(pos1), hi_min = min(pos0 + 1, cap), hi_max = min(pos1 + 1, cap);

    // The queries, 16 threads a row: read before the keys set out, since loads return in order; then scaled, their two
    // parts laid out as the operand that a lane reads.  Thread j holds the dims 32b + j and 32b + 16 + j (element 2m
    // + i of a block format's operand is dim 32b + 16i + 4g + m) or 32b + 2j and the next (binary16: element e is
    // 32b + 8g + e).
    uint32_t raw[RT][NB][2];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int r = min(16 * x + tid / 16, rows - 1), j = tid & 15, tok = token_of(row0 + r);
        const int64_t at = (w.first + tok) * a.ldq + (int64_t)(head * a.group + row0 + r - tok * a.group) * kDim;
        if (a.qtype == kF32) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) raw[x][b][i] = ((const uint32_t*)a.q)[at + 32 * b + (kKeyBlocks ? 16 * i + j : 2 * j + i)];
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) raw[x][b][i] = ((const uint16_t*)a.q)[at + 32 * b + (kKeyBlocks ? 16 * i + j : 2 * j + i)];
        }
    }

    // This wave's steps of the piece, those that the tile sees.
    int s0 = from, s1 = min(from + count, w.steps);
    s0 = max(s0, (lo_min - w.base) / kAtStep);
    s1 = min(s1, (hi_max - w.base + kAtStep - 1) / kAtStep);  // (hi_max below 0: none)
    const int ksteps = s1 > s0 + wave ? (s1 - s0 - wave + kWaves - 1) / kWaves : 0;
    const int start = w.base + kAtStep * (s0 + wave);
    const Mix mix;
    // Lane 2 i + half: where the half's keys and values lie of step block + i, and how far their scales are from there.  A
    // block of 32 steps is read anew after 30, before the steps that set out then.  A position that does not exist is
    // read at page 0 and not seen.
    int block = 0, kfar = 0, vfar = 0;
    uint64_t krows = 0, vrows = 0, missing = 0;
    const auto read_pages = [&](int start_step) {
        const AttendArgs& b = launch_args();
        const int k = start_step + (lane >> 1), pos = start + kAtStep * kWaves * k + 16 * (lane & 1), size = b.p.page_size;
        block = start_step;
        int place;
        const int page = kv_page(b.p, w.seq, k < ksteps ? pos : -1, place);
        missing = __ballot(page < 0);
        krows = (uint64_t)b.k.base + max(page, 0) * b.k.stride + ((int64_t)head * size * Side<KT, NB>::kRow + place * Side<KT, NB>::kFactor);
        vrows = (uint64_t)b.v.base + max(page, 0) * b.v.stride + ((int64_t)head * size * Side<VT, NB>::kRow + place * Side<VT, NB>::kFactor);
        kfar = (size - place) * Side<KT, NB>::kFactor + place * Side<KT, NB>::kScale;
        vfar = (size - place) * Side<VT, NB>::kFactor + place * Side<VT, NB>::kScale;
    };
    const auto rows_of = [&](uint64_t rows, int i) {
        const uint64_t at = (uint64_t)(uint32_t)lane_of((int)(rows >> 32), i) << 32 | (uint32_t)lane_of((int)rows, i);
        return (const char*)(const __attribute__((address_space(1))) char*)at;  // (global: loads that LDS does not wait for)
    };
    char* const ring = lds + S::kQueries + wave * S::kRing;
    const std::conditional_t<kStaged, Stage<KT, NB>, Nothing> kstage(lane);
    const std::conditional_t<kValBlocks, Stage<VT, NB>, Nothing> vstage(lane);
    Keys<KT, NB> keys[2];
    const auto fetch_keys = [&](int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 2 * (k - block) + h;
            if constexpr (kStaged) kstage.fetch(lane, ring + k % kDepth * S::kKeys, h, rows_of(krows, i), lane_of(kfar, i));
            else keys[h].load(lane, rows_of(krows, i));
        }
    };
    // Of binary16 the next step's; after the last anything, so that this step's do not stay in registers through it.
    const auto next_keys = [&](int k) {
        if (k < ksteps) {
            fetch_keys(k);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (uint32_t& word : keys[h].w) asm("" : "=v"(word));
        }
    };
    const auto fetch_values = [&](int k, Values<VT, NB>& vals) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 2 * (k - block) + h;
            if constexpr (kValBlocks) vstage.fetch(lane, ring + kDepth * S::kKeys + k % kDepth * S::kVals, h, rows_of(vrows, i), lane_of(vfar, i));
            else vals.load(lane, h, rows_of(vrows, i));
        }
    };
    Values<VT, NB> vals;
    // Waves without a step look pages up too: the queries are there then whatever way the compiler follows, and it puts
    // no wait for them further on, which would wait for the keys and values that set out now.
    read_pages(0);
    if (ksteps > 0) {
        // (values first where the compiler waits for the keys: they are there when the keys are)
        if constexpr (kStaged) fetch_keys(0);
        if constexpr (kValBlocks) fetch_values(0, vals);
        if constexpr (!kStaged) fetch_keys(0);
    }

#pragma unroll
    for (int x = 0; x < RT; ++x) {
        if (kWaves > 4 && wave >= 4) break;
        const int r = 16 * x + tid / 16, j = tid & 15;
        float v[NB][2], most = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = a.qtype == kF32 ? __builtin_bit_cast(float, raw[x][b][i]) : a.qtype == kBin16 ? h2f(raw[x][b][i]) : bf2f(raw[x][b][i]);
                v[b][i] = r < rows ? f * a.scale : 0.0f;
                most = __builtin_fmaxf(most, __builtin_fabsf(v[b][i]));
            }
        most = __builtin_fmaxf(most, dpp<0xB1>(most));
        most = __builtin_fmaxf(most, dpp<0x4E>(most));
        most = __builtin_fmaxf(most, dpp<0x141>(most));
        most = __builtin_fmaxf(most, dpp<0x140>(most));
        // the power of two that puts the largest in [2^13, 2^14); rows of nothing but tiny values stay what they are
        const int e = min(max((int)(__builtin_bit_cast(uint32_t, most) >> 23), 40), 254) - 126;
        const float up = power(14 - e);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t hi, lo;
            two_parts(mix, v[b][0] * up, v[b][1] * up, hi, lo);
            lq[x][b][0][16 * (j / 4) + r % 16][j % 4] = hi;
            lq[x][b][1][16 * (j / 4) + r % 16][j % 4] = lo;
        }
        if (j == 0) lc[r] = power(e - 14 + 2 + (kKeyBlocks ? 10 : 0));
    }
    if (kStaged && kDepth > 1 && ksteps > 1) {
        fetch_keys(1);
        fetch_values(1, vals);
    }
    __syncthreads();

    int rlo[RT], rhi[RT];
    float c[RT];  // scores are c times the sums of the scaled operands
    float4_t o[RT][kTiles];
    float m[RT], l[RT];
    // The folds of the blocks of values, the upper halves of two binary32 a dword; and for each of the lane's parts of a step's
    // scales the binary16 bits up to which there is room under every row's.
    constexpr int kPairs = Values<VT, NB>::kPairs;
    uint32_t fold[RT][kPairs];
    constexpr int kParts = (4 * NB + 15) / 16;
    u16x2 room[kParts];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int r = 16 * x + n;
        const int pos = w.len - w.n + token_of(row0 + min(r, rows - 1));  // (a row that does not exist sees what the last one does)
        rlo[x] = low(pos);
        rhi[x] = min(pos + 1, cap);
        c[x] = lc[r];
        m[x] = -INFINITY;
        l[x] = 0.0f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) fold[x][i] = 0x10001u * (kFoldMost >> 16);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[x][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) room[i] = u16x2{0, 0};
    const auto fold_bits = [&](int x, int b) { return b & 1 ? fold[x][b / 2] & 0xFFFF0000u : fold[x][b / 2] << 16; };
    const auto queries = [&](int x, int b, int part) { return __builtin_bit_cast(half8_t, *(const u32x4*)lq[x][b][part][lane]); };

    for (int k = 0; k < ksteps; ++k) {
        const int j0 = start + kAtStep * kWaves * k;
        int there = lane;  // where registers are short, the addresses in LDS are found anew rather than kept
        if constexpr (NB * RT >= 6) asm volatile("" : "+v"(there));
        if (k - block == 30) read_pages(k);
        const bool exist[2] = {!(missing >> (2 * (k - block)) & 1), !(missing >> (2 * (k - block) + 1) & 1)};
        if constexpr (kStaged) {
            // Behind this step's keys: its values, and the keys and values of the steps that have set out since.
            if (kDepth > 1 && k + 1 < ksteps) arrived<2 * Stage<VT, NB>::kLoads + Stage<KT, NB>::kLoads>();
            else arrived<Stage<VT, NB>::kLoads>();
#pragma unroll
            for (int h = 0; h < 2; ++h) keys[h].read(there, h, ring + k % kDepth * S::kKeys);
        } else if constexpr (kValBlocks) {
            arrived<0>();
        } else {
            fetch_values(k, vals);
        }
        float z[RT][8];
        {
            typename Keys<KT, NB>::Ready ready[2];
            keys[0].ready(ready[0]);
            keys[1].ready(ready[1]);
            float4_t s[RT][2], t[RT][2];
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[x][h] = t[x][h] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int r = 0; r < 4; ++r) z[x][4 * h + r] = 0.0f;
                }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (kKeyBlocks) __builtin_amdgcn_sched_barrier(0);
                const half8_t kb[2] = {Keys<KT, NB>::block(ready[0], b), Keys<KT, NB>::block(ready[1], b)};
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    const half8_t qh = queries(x, b, 0), ql = queries(x, b, 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (kKeyBlocks) {
                            float4_t u = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], ql, float4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
                            u = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], qh, u, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < 4; ++r) z[x][4 * h + r] = __builtin_fmaf(u[r], keys[h].scale(r, b), z[x][4 * h + r]);
                        } else {
                            s[x][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], qh, s[x][h], 0, 0, 0);
                            t[x][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], ql, t[x][h], 0, 0, 0);
                        }
                    }
                }
            }
            if constexpr (!kKeyBlocks) {
                bool odd = false;
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        z[x][i] = s[x][i / 4][i & 3] + t[x][i / 4][i & 3];
                        if (i & 1) odd |= __builtin_isunordered(z[x][i - 1], z[x][i]);
                    }
                // A key's infinity times the second part of a query's value, zero or of the other sign, would make NaN of the
                // infinity that the first part gives: there the second parts meet the finite values alone.  (The keys are read
                // again, a block at a time, so that they need no registers here where they are finite.)
                if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const char* rows_h = rows_of(krows, 2 * (k - block) + h);
                        float4_t u[RT], v[RT];
#pragma unroll
                        for (int x = 0; x < RT; ++x) u[x] = v[x] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            u32x4 kb;
                            Keys<KT, NB>::load_block(kb, lane, rows_h, b);
                            const u32x4 fin = {finite_halves(kb.x), finite_halves(kb.y), finite_halves(kb.z), finite_halves(kb.w)};
#pragma unroll
                            for (int x = 0; x < RT; ++x) {
                                u[x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, kb), queries(x, b, 0), u[x], 0, 0, 0);
                                v[x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, fin), queries(x, b, 1), v[x], 0, 0, 0);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
#pragma unroll
                        for (int x = 0; x < RT; ++x)
#pragma unroll
                            for (int r = 0; r < 4; ++r) z[x][4 * h + r] = u[x][r] + v[x][r];
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kStaged) {
            taken();
            if (k + kDepth < ksteps) fetch_keys(k + kDepth);
        } else if constexpr (kEarly) {
            if (kValBlocks && k + 1 < ksteps) {
                taken();
                fetch_values(k + 1, vals);
            }
            next_keys(k + 1);
        }
        // Positions that some row of the tile does not see: their scores go, whatever they are.  (The empty asm keeps
        // this a branch that steps in the middle of a cache skip.)
        const bool masked = j0 < lo_max || j0 + kAtStep > hi_min || !exist[0] || !exist[1];
        int seen[RT];  // bit i: position i of z
        if (masked) {
            asm volatile("");
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                seen[x] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool in = exist[i >> 2] && j >= rlo[x] && j < rhi[x];
                    seen[x] |= in ? 1 << i : 0;
                    z[x][i] = in ? z[x][i] : -INFINITY;
                }
            }
        }
        float top[RT];
        bool grew = false;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            top[x] = m[x];
#pragma unroll
            for (int i = 0; i < 8; ++i) top[x] = __builtin_fmaxf(top[x], z[x][i]);
            top[x] = rows_max(top[x]);
            grew |= top[x] > m[x];
        }
        if (__any(grew)) {
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                const float shrink = top[x] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[x] - top[x]) * c[x]);
                m[x] = top[x];
                l[x] *= shrink;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) o[x][t] *= shrink;
            }
        }
        // Weights: of binary16 values times 2^14; of blocks' to be multiplied by the scales and a power of two that
        // keeps the largest product there.
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const float from = m[x] == -INFINITY ? 0.0f : __builtin_fmaf(-m[x], c[x], kValBlocks ? 0.0f : 14.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[x][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[x][i], c[x], from));
                l[x] += z[x][i];
            }
        }
        if constexpr (kStaged) {
            // Behind this step's values: the keys and values that have set out since.
            constexpr int kK = Stage<KT, NB>::kLoads, kV = Stage<VT, NB>::kLoads;
            if (k + kDepth < ksteps) arrived<kDepth * kK + (kDepth - 1) * kV>();
            else if (kDepth > 1 && k + 1 < ksteps) arrived<kK + kV>();
            else arrived<0>();
        }
        if constexpr (kValBlocks) {
            vals.read(there, ring + kDepth * S::kKeys + k % kDepth * S::kVals);
        }
        if constexpr (kValBlocks) {
            vals.keep_words();
            char* const scales = ring + kDepth * S::kKeys + k % kDepth * S::kVals;
            // Scales that some row's folds leave no room for, seen or not: seldom after the first step.
            u16x2 part[kParts];
            Stage<VT, NB>::parts(scales, there & 15, there >> 4, part);
            if (__any(Stage<VT, NB>::above(part, room))) {
                asm volatile("");
                vals.keep_words();
                // The blocks' largest scales that each row sees.
                u16x2 most[RT][kPairs];
                const auto look = [&]() {
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        if (masked) {
                            vals.template largest<true>(seen[x], most[x]);
                        } else if (x > 0) {
#pragma unroll
                            for (int i = 0; i < kPairs; ++i) most[x][i] = most[0][i];
                        } else if constexpr (Stage<VT, NB>::kWhole) {
                            Stage<VT, NB>::largest(part, most[0]);
                        } else {
                            vals.template largest<false>(0, most[0]);
                        }
                    }
                };
                look();
                // A scale that is not finite must not meet the weight 0 of a row that does not see it: it is left
                // out, and makes its block NaN in the rows that do.
                u16x2 finite[kParts];
                int odd[RT];
                bool any_odd = false;
#pragma unroll
                for (int i = 0; i < kParts; ++i) finite[i] = u16x2{0x7BFF, 0x7BFF};
                if (__builtin_expect(__any(Stage<VT, NB>::above(part, finite)), 0)) {
                    any_odd = true;
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        odd[x] = 0;
#pragma unroll
                        for (int b = 0; b < NB; ++b) odd[x] |= most[x][b / 2][b % 2] >= 0x7C00 ? 1 << b : 0;
                    }
                    Stage<VT, NB>::keep_finite(scales, there);
                    vals.read_scales(there, scales);
                    Stage<VT, NB>::parts(scales, there & 15, there >> 4, part);
                    look();
                }
                uint32_t was[RT][kPairs];
                u16x2 least[kPairs];
#pragma unroll
                for (int i = 0; i < kPairs; ++i) least[i] = u16x2{0x7BFF, 0x7BFF};
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        uint32_t now[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // (a zero's is beyond kFoldMost)
                            const uint32_t scale = __builtin_bit_cast(uint32_t, h2f(most[x][i][e]));
                            now[e] = min(((127u + 13u + 127u) << 23) - (scale & 0x7F800000u), fold_bits(x, 2 * i + e));
                        }
                        was[x][i] = fold[x][i];
                        fold[x][i] = now[0] >> 16 | now[1];
                        const u16x2 limit = __builtin_bit_cast(u16x2, __builtin_convertvector((float2_t{over<15>(now[0]), over<15>(now[1])}), half2_t));
                        least[i] = __builtin_elementwise_min(least[i], limit - u16x2{1, 1});
                    }
                if (k > 0 || any_odd) {  // (the first step's sums are zeros)
#pragma unroll
                    for (int x = 0; x < RT; ++x)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint32_t old = b & 1 ? was[x][b / 2] & 0xFFFF0000u : was[x][b / 2] << 16;
                            float up = __builtin_bit_cast(float, fold_bits(x, b) - old + (127u << 23));
                            if (any_odd && odd[x] >> b & 1) up = NAN;
                            o[x][2 * b] *= up;
                            o[x][2 * b + 1] *= up;
                        }
                }
                // (the first step's rows are alike where they all see all of it)
                if (masked || k > 0) {
#pragma unroll
                    for (u16x2& v : least) v = min16_pair(v);
                }
                Stage<VT, NB>::share(there & 15, least, room);
                if constexpr (NB * RT > 4) {  // (their registers go to the sums)
                    asm volatile("" ::: "memory");
                    vals.read_scales(there, scales);
                }
                vals.keep_words();
            }
            vals.keep_words();
        } else {
            // Places that no row sees count as zeros.  Infinities and NaN must not meet the zeros of rows that do not see
            // them in the products, nor a weight's second part, zero or of the other sign: they are added one position at a
            // time, and left out there.
            if (masked) {
                asm volatile("");
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool some = exist[i >> 2] && j >= lo_min && j < hi_max;
#pragma unroll
                    for (int e = 0; e < Values<VT, NB>::kWords; ++e) vals.w[i][e] = some ? vals.w[i][e] : 0u;
                }
            }
            if (__builtin_expect(__any(vals.any_odd()), 0)) {
                if (!masked) {
#pragma unroll
                    for (int x = 0; x < RT; ++x) seen[x] = 0xFF;
                }
                float* weight = (float*)(lds + S::kQueries + wave * S::kOdd);
                uint32_t* row = (uint32_t*)(weight + kRows * kAtStep);
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) weight[(16 * x + n) * kAtStep + 16 * (i >> 2) + 4 * g + (i & 3)] = seen[x] >> i & 1 ? z[x][i] : -1.0f;
                for (int u = 0; u < kAtStep; ++u) {
                    if (g == u / 4 % 4) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i == 4 * (u / 16) + u % 4)
#pragma unroll
                                for (int e = 0; e < Values<VT, NB>::kWords; ++e) row[n * Values<VT, NB>::kWords + e] = vals.w[i][e];
                    }
                    wave_fence();
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        const float p = weight[(16 * x + n) * kAtStep + u];
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const uint32_t v = ((const uint16_t*)row)[Values<VT, NB>::dim(t, 4 * g + r)];
                                if (p >= 0.0f && not_finite(v)) o[x][t][r] += p * h2f(v);
                            }
                    }
                    wave_fence();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < Values<VT, NB>::kWords; ++e) vals.w[i][e] = finite_halves(vals.w[i][e]);
            }
        }
        // The sums of values.
        typename Values<VT, NB>::Ready ready;
        vals.ready(ready);
        half8_t ph[RT], pl[RT];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            if (kValBlocks ? t % 2 == 0 : t == 0) {
                if constexpr (kValBlocks) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    uint32_t hi[4], lo[4];
                    if constexpr (kValBlocks) {
                        const float f = __builtin_bit_cast(float, fold_bits(x, t / 2));
                        float u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = z[x][i] * f;
                        scaled_parts(mix, u, [&](int i) { return vals.scale(i, t / 2); }, hi, lo);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) two_parts(mix, z[x][2 * i], z[x][2 * i + 1], hi[i], lo[i]);
                    }
                    ph[x] = as_half8(hi[0], hi[1], hi[2], hi[3]);
                    pl[x] = as_half8(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            const half8_t v = Values<VT, NB>::tile(ready, t);
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                o[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl[x], o[x][t], 0, 0, 0);
                o[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph[x], o[x][t], 0, 0, 0);
            }
        }
        if constexpr (kStaged) {
            taken();
            if (k + kDepth < ksteps) fetch_values(k + kDepth, vals);
        } else if constexpr (!kEarly) {
            if (kValBlocks && k + 1 < ksteps) {
                taken();
                fetch_values(k + 1, vals);
            }
            next_keys(k + 1);
        }
    }

    // The waves' results, in base-2 units of the scores, to LDS; then four dims of a row a lane.
    const int active = min(kWaves, max(s1 - s0, 1));  // waves with a step (one at least: the zeros of none)
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        l[x] = rows_sum(l[x]) * (kValBlocks ? 1.0f : power(-14));
        m[x] *= c[x];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[x][t] *= kValBlocks ? over<10>(fold_bits(x, t / 2)) : power(-14);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        if (wave >= active || 16 * x + n >= rows) continue;
        if (g == 0) {
            lm[wave][16 * x + n] = m[x];
            ll[wave][16 * x + n] = l[x];
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) so[wave][16 * x + n][Values<VT, NB>::dim(t, 4 * g + r)] = o[x][t][r];
    }
    __syncthreads();
    const AttendArgs& b = launch_args();
    float* part = b.parts + ((int64_t)slot * b.p.nheads + head) * part_floats(kRows, kDim);
    for (int i = tid; i < rows * (kDim / 4); i += 64 * kWaves) {
        const int r = i / (kDim / 4), d = 4 * (i - r * (kDim / 4));
        float most = -INFINITY, sum = 0.0f;
        float4_t f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int y = 0; y < kWaves; ++y) most = y < active ? __builtin_fmaxf(most, lm[y][r]) : most;
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
            if (y >= active) break;
            const float weight = beside(lm[y][r], most);
            sum += weight * ll[y][r];
            f += weight * *(const float4_t*)&so[y][r][d];
        }
        if (slot < 0) {
            f *= sum != 0.0f ? 1.0f / sum : 0.0f;
            write_row(b, w.first, head, row0 + r, d, f, most, sum);
        } else {
            if (d == 0) {
                part[r] = most;
                part[kRows + r] = sum;
            }
            *(float4_t*)(part + 2 * kRows + r * kDim + d) = f;
        }
    }
}

template <int KT, int VT, int NB, int RT>
__global__ __launch_bounds__((64 * Shape<KT, VT, NB, RT>::kWaves), 2) void attend_kernel(AttendArgs) {
    const AttendArgs& a = launch_args();
    using S = Shape<KT, VT, NB, RT>;
    constexpr int kRows = 16 * RT, kDim = 32 * NB;
    __shared__ __attribute__((aligned(16))) char lds[S::kBytes];
    __shared__ float lc[kRows];
    uint32_t head;
    int run = (int)kv_divide(blockIdx.x, a.p.nheads, a.p.per_head, head);
    SeqWork mine;
    const Split split = find_split(a, kRows, mine);
    if (split.paired) {
        const int half = (a.target + 1) / 2;
        run = run < half ? 2 * run : 2 * (run - half) + 1;
    }
    const int begin = split.begin(run), end = min(split.begin(run + 1), split.all);
    const bool tells = a.pieces && head == 0 && threadIdx.x == 0;
    if (tells) a.pieces[2 * run].count = a.pieces[2 * run + 1].count = 0;
    for (int at = begin; at < end;) {
        if (at > begin && !a.plan) mine = lane_work(a, threadIdx.x & 63, kRows);  // (not kept beside the sums)
        const Tile tl = find_tile(a, split, at, kRows, mine);
        const SeqWork& w = tl.w;
        const int piece = at - tl.at, units = min(end - tl.at, tl.live) - piece;
        at = tl.at + tl.units;
        if (units <= 0) continue;
        int slot = -1;
        if (units != tl.live) {
            // The second of the two, if the tile begins here.
            const Per per(split.pair);
            const int from = split.run_of(per, tl.at);
            slot = 2 * run + (run == from ? 1 : 0);
            if (tells) a.pieces[slot] = Piece{split.run_of(per, tl.at + tl.live - 1) - from + 1, run - from, w.first, tl.tile << 6 | min(kRows, w.n * a.group - tl.tile * kRows)};
        }
        attend_piece<KT, VT, NB, RT>(w, tl.tile, piece << a.shift, units << a.shift, lds, lc, (int)head, slot);
        __syncthreads();
    }
}

template <int KT, int VT, int NB, int RT>
void attend_launch(const AttendArgs& a, unsigned grid, hipStream_t st) {
    hipLaunchKernelGGL((attend_kernel<KT, VT, NB, RT>), dim3(grid), dim3(64 * Shape<KT, VT, NB, RT>::kWaves), 0, st, a);
}

// The launch of one pair of formats, instantiated in a source of its own per format of the keys.
template <int KT, int VT>
void attend_pair(const AttendArgs& a, unsigned grid, int rt, hipStream_t st) {
    switch (a.p.dim / 32 * 2 + rt) {
        case 5: attend_launch<KT, VT, 2, 1>(a, grid, st); break;
        case 6: attend_launch<KT, VT, 2, 2>(a, grid, st); break;
        case 7: attend_launch<KT, VT, 3, 1>(a, grid, st); break;
        case 8: attend_launch<KT, VT, 3, 2>(a, grid, st); break;
        case 9: attend_launch<KT, VT, 4, 1>(a, grid, st); break;
        case 10: attend_launch<KT, VT, 4, 2>(a, grid, st); break;
        case 13: attend_launch<KT, VT, 6, 1>(a, grid, st); break;
        default: attend_launch<KT, VT, 8, 1>(a, grid, st); break;
    }
}
void attend_f16(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);
void attend_q8(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);
void attend_iq4(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);

}  // namespace qmm
