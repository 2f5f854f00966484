// qmm_attend.hip -- attention of new tokens over the paged key-value cache: the split of many sequences, the
// join of a split one and the entry point, for gfx950.  The pass itself is in qmm_attend.h.
#include "qmm_attend.h"

namespace qmm {

// The split of more sequences than a wave looks through: lengths, all, then the units before each sequence.
__global__ __launch_bounds__(1024) void attend_plan_kernel(AttendArgs a, int rows, int32_t* plan) {
    __shared__ int tokens[16], units[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nseq = a.p.nseq;
    int64_t all = 0;
    int before = 0;
    for (int s0 = 0; s0 < nseq; s0 += 1024) {
        const int s = s0 + threadIdx.x;
        const SeqWork w = lane_work(a, s, rows);
        const int mine = w.tiles * line_units(a, w.steps), upto = wave_scan(mine), n = wave_total(w.n);
        __syncthreads();
        if (lane == 63) {
            units[wave] = upto;
            tokens[wave] = n;
        }
        __syncthreads();
        int off = before;
        for (int i = 0; i < 16; ++i) {
            off += i < wave ? units[i] : 0;
            before += units[i];
            all += tokens[i];
        }
        if (s < nseq) plan[3 + s] = off + upto - mine;
    }
    const Split split = line_split(a, before, 0, all, [&](int) { return 0x3FFFFFFF; });
    if (threadIdx.x == 0) {
        plan[0] = split.pair;
        plan[1] = split.first;
        plan[2] = split.all;
        plan[3 + nseq] = before;
    }
}

// The pieces of a tile joined, in their order, by as many workgroups as it has pieces: they share the tile's groups of
// four dims.  A group's pieces go to E lanes of a wave, each every E-th of them, lanes of neighbouring groups
// beside each other.  Bound: two loads one after the other (what the pass told, the pieces): 4 us, 2.5 at least.
template <int E>
__device__ __forceinline__ void join(const AttendArgs& a, const Piece& t, int run, int head, int tile_rows) {
    const int dim = a.p.dim, row0 = (t.rows >> 6) * tile_rows, rows = t.rows & 63, quads = rows * (dim / 4), from = run - t.mine;
    const int lane = threadIdx.x & 63, turn = lane / (64 / E);
    const int64_t size = part_floats(tile_rows, dim);
    for (int u = (t.mine * 4 + (int)(threadIdx.x >> 6)) * (64 / E); u < quads; u += t.count * 4 * (64 / E)) {
        const int at = min(u + lane % (64 / E), quads - 1), r = at / (dim / 4), d = 4 * (at - r * (dim / 4));
        float most = -INFINITY, sum = 0.0f;
        float4_t f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int i = turn; i < t.count; i += E) {
            const float* p = a.parts + ((int64_t)(2 * (from + i) + (i ? 0 : 1)) * a.p.nheads + head) * size;
            const float m = p[r], l = p[tile_rows + r];
            const float4_t o = *(const float4_t*)(p + 2 * tile_rows + r * dim + d);
            const float now = __builtin_fmaxf(most, m), old = beside(most, now), fresh = beside(m, now);
            most = now;
            sum = sum * old + l * fresh;
            f = f * old + o * fresh;
        }
#pragma unroll
        for (int x = 64 / E; x < 64; x <<= 1) {
            const float m = __shfl_xor(most, x, 64), l = __shfl_xor(sum, x, 64);
            const float now = __builtin_fmaxf(most, m), old = beside(most, now), fresh = beside(m, now);
            most = now;
            sum = sum * old + l * fresh;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = f[e] * old + __shfl_xor(f[e], x, 64) * fresh;
        }
        if (turn == 0 && u + lane < quads) {
            f *= sum != 0.0f ? 1.0f / sum : 0.0f;
            write_row(a, t.first, head, row0 + r, d, f, most, sum);
        }
    }
}

// The workgroup's piece of a tile that began before it, then of one that begins there (seldom both).
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int tile_rows) {
    uint32_t head;
    const int run = (int)kv_divide(blockIdx.x, a.p.nheads, a.p.per_head, head);
    const Piece both[2] = {a.pieces[2 * run], a.pieces[2 * run + 1]};
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const Piece t = i ? both[1] : both[0];
        if (t.count == 0) continue;
        // As few pieces a lane as leave a lane to every group at once (32 x 256 wide, 16 rows: 28 us, with 8 lanes a group 31).
        const int room = 256 * t.count, quads = (t.rows & 63) * (a.p.dim / 4);
        if (t.count >= 16 && room >= 16 * quads) join<16>(a, t, run, (int)head, tile_rows);
        else if (t.count >= 8 && room >= 8 * quads) join<8>(a, t, run, (int)head, tile_rows);
        else if (t.count >= 4 && room >= 4 * quads) join<4>(a, t, run, (int)head, tile_rows);
        else if (room >= 2 * quads) join<2>(a, t, run, (int)head, tile_rows);
        else join<1>(a, t, run, (int)head, tile_rows);
    }
}

}  // namespace qmm

#include <algorithm>

#include "qmm_kv_host.h"

using namespace qmm;

namespace {

constexpr int kAtCus = 256;
// Workgroups run two on a CU, but for keys and values of q8_0 that are 256 wide, whose eight waves take the LDS of a whole
// one (8 x 4096: 25 us, split for two a CU, one after the other, 33; 64 of up to 1500: 39, 34).
static_assert(Shape<kKvQ8, kKvQ8, 8, 1>::kWaves == 8 && Shape<kKvQ8, kKvIq4, 8, 1>::kWaves == 4 && Shape<kKvF16, kKvQ8, 8, 1>::kWaves == 4 &&
              Shape<kKvQ8, kKvQ8, 6, 1>::kWaves == 4 && Shape<kKvQ8, kKvQ8, 4, 2>::kWaves == 4, "as attend_shape counts them");
constexpr int kAtLeast = 8;     // steps that a tile counts for at least on the line

struct AttendShape {
    KvPlace p;
    int rt;          // 16-row tiles a workgroup
    int target;      // workgroups a head of keys, at most
    int shift;       // 2^shift steps are a unit of the split
    bool split;      // a tile can have more than one piece
    size_t bytes;    // of the workspace: pieces, what is told of them, the plan
    size_t told, plan;  // their offsets
};

int attend_shape(AttendShape& s, const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                 const int32_t* lens, const int32_t* seg_off, int nseq, int64_t ntok, int nheads) {
    const int rc = kv_place(s.p, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok);
    if (rc != QMM_OK) return rc;
    if (nheads < 1 || nheads % c->nheads) return QMM_EINVAL;
    if (nheads > 1024 || ntok * nheads > kKvMaxRows || kv_row_bytes(c->vtype, 64) > kv_row_bytes(c->ktype, 64)) return QMM_EUNSUPPORTED;
    const int64_t group = nheads / c->nheads;
    // 32 rows a workgroup where sequences have more than 16 on average (32 x 4096 q8_0, 32 heads a head of keys: 53 us, 61
    // by 16; 8 tokens of 5, binary16: 42, 68).  Two tiles of wider heads do not fit the registers.
    const bool wide = c->head_dim <= 128;
    s.rt = wide && nseq && group * ((ntok + nseq - 1) / nseq) > 16 ? 2 : 1;
    // At most this many steps a tile (a walk may begin 15 positions early), and so workgroups with a length of the line.
    const bool alone = c->ktype == QMM_Q8_0 && c->vtype == QMM_Q8_0 && c->head_dim == 256;
    const int64_t steps = (max_pages * c->page_size + kAtStep - 1) / kAtStep + 1;
    const auto tiles_of = [&](int64_t rows) { return std::min(nseq + ntok * group / rows, ntok * ((group + rows - 1) / rows)); };
    const auto target_of = [&](int64_t tiles) {
        return (int)std::max(std::min((int64_t)((alone ? 1 : 2) * kAtCus / c->nheads), tiles * ((steps + kAtWaves - 1) / kAtWaves)), (int64_t)1);
    };
    const int64_t tiles = tiles_of(16 * s.rt), most = tiles_of(16);
    s.target = target_of(tiles);
    for (s.shift = 0; (tiles * std::max(steps, (int64_t)kAtLeast)) >> s.shift > 1 << 29;) ++s.shift;
    const int whole = nseq > kAtInline ? kAtWaves : tiles * c->nheads >= kAtCus ? kAtShort : kAtShort / 2;
    s.split = steps > whole || tiles > s.target;
    if (!s.split) s.target = (int)std::max(tiles, (int64_t)1);
    // The size for tiles of 16 rows, which are more, and of 32, which are larger: what is enough for a call is enough for
    // smaller ones, of whatever proportions.
    const int room = target_of(most);
    const bool pieces = steps > kAtWaves || most > room;
    s.told = pieces ? (size_t)(2 * room * c->nheads * part_floats(wide ? 32 : 16, c->head_dim) * 4) : 0;
    s.plan = s.told + (pieces ? 2 * room * sizeof(Piece) : 0);
    s.bytes = s.plan + (nseq > kAtInline ? (size_t)(nseq + 4) * 4 : 0);
    s.bytes = s.bytes < 16 ? 16 : s.bytes;
    return QMM_OK;
}

}  // namespace

extern "C" size_t qmm_kv_attend_workspace(const qmm_kv_cache* c, int64_t ntok, int nheads, int nseq, int64_t max_pages) {
    AttendShape s;
    static const int32_t some = 0;
    return attend_shape(s, c, &some, max_pages, max_pages, &some, &some, nseq, ntok, nheads) == QMM_OK ? s.bytes : 0;
}

extern "C" int qmm_kv_attend(const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                             const int32_t* seg_off, int nseq, int qtype, const void* q, int64_t ldq, int64_t ntok, int nheads,
                             float scale, int64_t window, int otype, void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
    if (!valid_type(qtype) || !valid_type(otype) || window < 0 || !(scale >= -3.4e38f) || !(scale <= 3.4e38f)) return QMM_EINVAL;
    AttendShape s;
    const int rc = attend_shape(s, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok, nheads);
    if (rc != QMM_OK) return rc;
    const int64_t width = (int64_t)nheads * c->head_dim;
    if (ldq < width || ldo < width) return QMM_EINVAL;
    if (ntok == 0 || nseq == 0) return QMM_OK;
    if (!q || !out || !ws) return QMM_EINVAL;
    if (!aligned(q, type_bytes(qtype)) || !aligned(out, type_bytes(otype)) || !aligned(lse, 4) || !aligned(ws, 16)) return QMM_EALIGN;
    if (ws_bytes < s.bytes) return QMM_ESPACE;
    if (out == q) return QMM_EINVAL;
    const auto fours = [](const void* p, int64_t ld, int type) { return aligned(p, 4 * type_bytes(type)) && ld % 4 == 0; };
    AttendArgs a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.parts = (float*)ws;
    a.pieces = s.split ? (Piece*)((char*)ws + s.told) : nullptr;
    a.plan = nseq > kAtInline ? (const int32_t*)((char*)ws + s.plan) : nullptr;
    a.ldq = ldq;
    a.ldo = ldo;
    a.k = KvSide{(char*)c->k, c->kstride, c->ktype};
    a.v = KvSide{(char*)c->v, c->vstride, c->vtype};
    a.p = s.p;
    a.nheads = nheads;
    a.group = nheads / c->nheads;
    a.per_group = kv_per(a.group);
    a.qtype = qtype;
    a.otype = otype;
    a.scale = (float)((double)scale * (1.4426950408889634 / 4));
    a.window = (int)std::min(window, (int64_t)0x7FFFFFFF);  // more than any position
    a.target = s.target;
    a.one = std::max(kAtCus / c->nheads, 1);
    a.shift = s.shift;
    a.per_target = kv_per(a.target);
    a.least = kAtLeast;
    a.vec = fours(out, ldo, otype);
    const hipStream_t st = as_stream(stream);
    if (a.plan) hipLaunchKernelGGL(attend_plan_kernel, dim3(1), dim3(1024), 0, st, a, 16 * s.rt, const_cast<int32_t*>(a.plan));
    const unsigned grid = (unsigned)(s.target * c->nheads);
    if (c->ktype == QMM_F16) attend_f16(a, grid, s.rt, st);
    else if (c->ktype == QMM_Q8_0) attend_q8(a, grid, s.rt, st);
    else attend_iq4(a, grid, s.rt, st);
    if (s.split) hipLaunchKernelGGL(attend_join_kernel, dim3(grid), dim3(256), 0, st, a, 16 * s.rt);
    return launch_status();
}
