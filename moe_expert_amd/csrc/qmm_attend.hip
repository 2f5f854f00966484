// qmm_attend.hip -- attention of new tokens over the paged key-value cache: the split of many sequences, the
// join of a split one and the entry point, for gfx950.  The pass itself is in qmm_attend.h.
#include "qmm_attend.h"

namespace qmm {

// The split of more sequences than a wave's registers hold: items and slots before each sequence.
__global__ __launch_bounds__(1024) void attend_plan_kernel(AttendArgs a, int rows, int32_t* plan) {
    __shared__ int64_t work[16];
    __shared__ int items[16], slots[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nseq = a.p.nseq;
    int64_t sum = 0;
    for (int s = threadIdx.x; s - lane < nseq; s += 1024) {
        const SeqWork w = lane_work(a, s, rows);
        const int64_t mine = (int64_t)w.steps * w.tiles;
        sum += ((int64_t)wave_total((int)(mine >> 24)) << 24) + wave_total((int)(mine & 0xFFFFFF));
    }
    if (lane == 0) work[wave] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < 16; ++i) sum += work[i];
    const int c = part_steps(a, sum, [&](int) { return a.target + 1; });
    int before = 0, sbefore = 0;
    for (int s0 = 0; s0 < nseq; s0 += 1024) {
        const int s = s0 + threadIdx.x;
        int mine = 0, slot = 0;
        if (s < nseq) {
            const SeqWork w = seq_work(a, s, rows);
            const int parts = parts_of(w, c);
            mine = parts * w.tiles;
            slot = parts > 1 ? mine : 0;
        }
        const int upto = wave_scan(mine), sl = wave_scan(slot);
        __syncthreads();
        if (lane == 63) {
            items[wave] = upto;
            slots[wave] = sl;
        }
        __syncthreads();
        int off = before, soff = sbefore;
        for (int i = 0; i < 16; ++i) {
            off += i < wave ? items[i] : 0;
            soff += i < wave ? slots[i] : 0;
            before += items[i];
            sbefore += slots[i];
        }
        if (s < nseq) {
            plan[1 + s] = off + upto - mine;
            plan[2 + nseq + s] = soff + sl - slot;
        }
    }
    if (threadIdx.x == 0) {
        plan[0] = c;
        plan[1 + nseq] = before;
        plan[2 + 2 * nseq] = sbefore;
    }
}

// The parts of a tile joined, in the order of the parts.  The tile's workgroups share its groups of four dims; a
// group's parts go to E lanes of a wave, each every E-th of them, lanes of neighbouring groups beside each other.
template <int E>
__device__ __forceinline__ void join(const AttendArgs& a, const Item& it, int head, int tile_rows) {
    const int dim = a.p.dim, row0 = it.tile * tile_rows, rows = min(tile_rows, it.w.n * a.group - row0), quads = rows * (dim / 4);
    const int lane = threadIdx.x & 63, run = lane / (64 / E);
    const int64_t step = a.p.nheads * part_floats(tile_rows, dim);
    const float* part = a.parts + ((int64_t)it.slot * a.p.nheads + head) * part_floats(tile_rows, dim);
    for (int u = (it.part * 4 + (int)(threadIdx.x >> 6)) * (64 / E); u < quads; u += it.parts * 4 * (64 / E)) {
        const int at = min(u + lane % (64 / E), quads - 1), r = at / (dim / 4), d = 4 * (at - r * (dim / 4));
        float most = -INFINITY, sum = 0.0f;
        float4_t f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int i = run; i < it.parts; i += E) {
            const float* p = part + i * step;
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
        if (run == 0 && u + lane < quads) {
            f *= sum != 0.0f ? 1.0f / sum : 0.0f;
            write_row(a, it.w.first, head, row0 + r, d, f, most, sum);
        }
    }
}

__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int tile_rows) {
    const int head = (int)(blockIdx.x % (uint32_t)a.p.nheads);
    Item it;
    if (!find_item(a, (int)(blockIdx.x / (uint32_t)a.p.nheads), tile_rows, it) || it.parts == 1) return;
    if (it.slot < 0 || it.slot + it.parts > a.slots) return;
    if (it.parts <= 16) join<1>(a, it, head, tile_rows);
    else join<16>(a, it, head, tile_rows);
}

}  // namespace qmm

#include <algorithm>

#include "qmm_kv_host.h"

using namespace qmm;

namespace {

constexpr int64_t kAtTarget = 512;  // workgroups to split the caches over: two for every CU, what runs at once
constexpr int kAtLeast = 8;          // steps of the shortest part

struct AttendShape {
    KvPlace p;
    int rt;          // 16-row tiles a workgroup
    int target, least;
    int64_t items;   // workgroups a head of keys, at most
    int64_t slots;   // parts of tiles that have several, at most
    size_t bytes;    // of the workspace: parts, then the plan
    size_t plan;     // its offset
};

int attend_shape(AttendShape& s, const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                 const int32_t* lens, const int32_t* seg_off, int nseq, int64_t ntok, int nheads) {
    const int rc = kv_place(s.p, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok);
    if (rc != QMM_OK) return rc;
    if (nheads < 1 || nheads % c->nheads) return QMM_EINVAL;
    if (nheads > 1024 || ntok * nheads > kKvMaxRows || kv_row_bytes(c->vtype, 64) > kv_row_bytes(c->ktype, 64)) return QMM_EUNSUPPORTED;
    const int64_t group = nheads / c->nheads;
    const bool wide = c->head_dim <= 128;  // two tiles of wider heads do not fit the registers
    s.rt = wide && nseq && group * ((ntok + nseq - 1) / nseq) > 16 ? 2 : 1;
    const int64_t rows = 16 * s.rt, tiles = std::min(nseq + ntok * group / rows, ntok * ((group + rows - 1) / rows));
    s.target = (int)std::max(kAtTarget / c->nheads, (int64_t)1);
    s.least = kAtLeast;
    const int64_t steps = (max_pages * c->page_size + kAtStep - 1) / kAtStep + 1, most = (steps + s.least - 1) / s.least;
    s.items = std::min(kAtRounds * s.target + tiles, tiles * most);
    s.slots = most > 1 ? std::min((int64_t)2 * kAtRounds * s.target, tiles * most) : 0;
    if (s.items * c->nheads >= 1 << 24) return QMM_EUNSUPPORTED;  // below 2^32 threads
    // (sized for 32 rows where a call of other proportions would take them)
    s.plan = (size_t)(s.slots * c->nheads * part_floats(wide ? 32 : 16, c->head_dim) * 4 + 15) & ~(size_t)15;
    s.bytes = s.plan + (nseq > kAtInline ? (size_t)(2 * nseq + 3) * 4 : 0);
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
    const auto fours = [](const void* p, int64_t ld, int type) { return aligned(p, 4 * type_bytes(type)) && ld % 4 == 0; };
    AttendArgs a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.parts = (float*)ws;
    a.plan = nseq > kAtInline ? (const int32_t*)((char*)ws + s.plan) : nullptr;
    a.ldq = ldq;
    a.ldo = ldo;
    a.k = KvSide{(char*)c->k, c->kstride, c->ktype};
    a.v = KvSide{(char*)c->v, c->vstride, c->vtype};
    a.p = s.p;
    a.nheads = nheads;
    a.group = nheads / c->nheads;
    a.qtype = qtype;
    a.otype = otype;
    a.scale = (float)((double)scale * 1.4426950408889634);
    a.window = (int)std::min(window, (int64_t)0x7FFFFFFF);  // more than any position
    a.target = s.target;
    a.least = s.least;
    a.slots = (int)s.slots;
    a.vec = fours(out, ldo, otype);
    const hipStream_t st = as_stream(stream);
    if (a.plan) hipLaunchKernelGGL(attend_plan_kernel, dim3(1), dim3(1024), 0, st, a, 16 * s.rt, const_cast<int32_t*>(a.plan));
    const unsigned grid = (unsigned)(s.items * c->nheads);
    if (c->ktype == QMM_F16) attend_f16(a, grid, s.rt, st);
    else if (c->ktype == QMM_Q8_0) attend_q8(a, grid, s.rt, st);
    else attend_iq4(a, grid, s.rt, st);
    if (s.slots) hipLaunchKernelGGL(attend_join_kernel, dim3(grid), dim3(256), 0, st, a, 16 * s.rt);
    return launch_status();
}
