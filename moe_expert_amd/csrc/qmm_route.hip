// qmm_route.hip -- routing of tokens to experts and the expert-sorted entry lists, for gfx950.
//
// Routing: s = softmax(l) or 1 / (1 + exp(-l)) in binary32, c = s + bias, the best topk of c (within
// the best runs of experts), weights s / sum of the chosen s.  Dispatch: a stable counting sort of the
// chosen (token, k) by expert.
#include "qmm_values.h"

namespace qmm {

constexpr int kRouteMaxExperts = 1024, kRouteMaxTopk = 64, kRouteMaxGroups = 64;

// LDS written by some lanes of a wave and read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t ldl, ntok;
    int ltype, nexperts, softmax, ngroups, topk_groups, group_top, topk, renorm;
    float scale;
    int32_t* ids;
    float* weights;
};

constexpr float kNever = -__builtin_inff();

// Maximum (of integers) and sum over aligned groups of L lanes (16, 32, 64), in every lane.
template <int L>
__device__ __forceinline__ int lanes_max(int v) {
    const auto larger = [](int a, int b) { return a > b ? a : b; };
    v = larger(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true));
    v = larger(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true));
    v = larger(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));
    v = larger(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = larger((int)r[0], (int)r[1]);
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = larger((int)r[0], (int)r[1]);
    }
    return v;
}

// Binary32 values (no NaN) as integers of the same order, -0 and +0 the same: maxima of integers need
// none of the canonicalising moves that float maxima do.
constexpr int kNeverKey = (int)0x80000000;  // below every value's
__device__ __forceinline__ int key_of(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int k) { return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7FFFFFFF)); }

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
    if constexpr (L >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

__device__ __forceinline__ float run_score(const RouteArgs& a, float best, float second) {
    return a.group_top == 1 ? best : second == kNever ? kNever : best + second;
}

// L lanes per token, V experts a lane: lane q holds experts q V .. q V + V - 1, so the lowest lane that
// holds a value holds the lowest expert.  Every token lives in one wave: the best choice is found topk
// times by a maximum over its lanes and a ballot of who holds it, with no barrier.  As few lanes as hold
// the row at 8 experts each (16 for more than 512), so a wave serves up to four tokens: 8192 tokens of
// 128 experts 5.2 us against 6.1 with 4 experts a lane (8 tokens: 4.4 against 3.9), of 256 7.3
// against 9.4 with 4 and 7.6 with 16.  VEC: rows in
// aligned pieces of 8 (V = 8 or 16).
// Bound: VALU and what a choice waits for: with 8 experts a lane 14 vector instructions find the best, 34
// locate and remove it, and some 25 scalar ones and no-ops stand between them; few tokens: that chain's
// latency.  8192 tokens, top-8 of 128: 5.2 us (4.7 MB; one token a wave with exchanges through lanes
// 17.4); 8 tokens 4.3 us; 8192 tokens, top-10 of 512 14 us; 4099 tokens of 256 experts in 8 runs with
// sigmoid and bias 9.3 us, in which each bias value is a load behind its own branch, waited for before
// the next, and scores are divided by a sum of 1.
template <int L, int V, bool VEC>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    constexpr int T = 256 / L;
    __shared__ float scores[T][L * V], runs[T][kRouteMaxGroups];
    __shared__ int chosen[T][kRouteMaxTopk];
    const int q = threadIdx.x % L, g = threadIdx.x / L, E = a.nexperts, e0 = q * V;
    const int64_t t = (int64_t)blockIdx.x * T + g;
    const bool live = t < a.ntok;  // lanes past the tokens go along on the last one and store nothing
    const int64_t row = (live ? t : a.ntok - 1) * a.ldl;
    float c[V], s[V];
    if constexpr (VEC) {
        const char* p = (const char*)a.logits + row * (a.ltype == kF32 ? 4 : 2);
        Raw8 raw[V / 8];
#pragma unroll
        for (int i = 0; i < V / 8; ++i) load_raw8(raw[i], p, e0 + 8 * i < E ? e0 + 8 * i : 0, a.ltype);
#pragma unroll
        for (int i = 0; i < V / 8; ++i) unpack8(raw[i], a.ltype, c + 8 * i);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = load_value(a.logits, row + (e0 + v < E ? e0 + v : 0), a.ltype);
    }
    float top = kNever;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (e0 + v >= E || c[v] != c[v]) c[v] = kNever;
        top = fmaxf(top, c[v]);
    }
    // s: a factor of the score (softmax: over the sum, known for the whole row) or the score
    float sum = 1.0f;
    if (a.softmax) {
        top = value_of(lanes_max<L>(key_of(top)));
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = c[v] == kNever ? 0.0f : c[v] == top ? 1.0f : expf(c[v] - top);
            sum += s[v];
        }
        sum = lanes_sum<L>(sum);
        if (sum == 0.0f) sum = 1.0f;  // no expert
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-c[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) scores[g][e0 + v] = s[v];
    if (!a.softmax || a.bias || (a.ngroups > 1 && a.group_top > 1)) {  // chosen by score, else by logit
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float sc = a.softmax ? s[v] / sum : s[v];
            const float d = a.bias ? sc + a.bias[e0 + v < E ? e0 + v : 0] : sc;
            c[v] = c[v] == kNever || d != d ? kNever : d;
        }
    }
    if (a.ngroups > 1) {
        // a run's score: by its lanes where it is a power of two of whole lanes, else from LDS
        const int per = E / a.ngroups, lanes = per / V;
        __shared__ float members[T][L * V];
        __shared__ int beaten[T][kRouteMaxGroups];
        float m0 = kNever, m1 = kNever;
        if (lanes * V == per && (lanes & (lanes - 1)) == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                m1 = fmaxf(m1, fminf(m0, c[v]));
                m0 = fmaxf(m0, c[v]);
            }
            for (int d = 1; d < lanes; d <<= 1) {
                const float o0 = __shfl_xor(m0, d, 64), o1 = __shfl_xor(m1, d, 64);
                m1 = fmaxf(fmaxf(m1, o1), fminf(m0, o0));
                m0 = fmaxf(m0, o0);
            }
            if (e0 < E && e0 % per == 0) runs[g][e0 / per] = run_score(a, m0, m1);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) members[g][e0 + v] = c[v];
            wave_sync();
            for (int r = q; r < a.ngroups; r += L) {
                m0 = m1 = kNever;
                for (int i = 0; i < per; ++i) {
                    const float x = members[g][r * per + i];
                    m1 = fmaxf(m1, fminf(m0, x));
                    m0 = fmaxf(m0, x);
                }
                runs[g][r] = run_score(a, m0, m1);
            }
        }
        wave_sync();
        // experts of a run that at least topk_groups others beat are out
        for (int r = q; r < a.ngroups; r += L) {
            const float mine = runs[g][r];
            int better = 0;
            for (int o = 0; o < a.ngroups; ++o) {
                const float x = runs[g][o];
                better += (int)(x > mine) | ((int)(x == mine) & (int)(o < r));
            }
            beaten[g][r] = better >= a.topk_groups;
        }
        wave_sync();
        int r = (e0 < E ? e0 : E - 1) / per, left = (r + 1) * per - e0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (v == left) {
                r = r + 1 < a.ngroups ? r + 1 : r;
                left += per;
            }
            c[v] = beaten[g][r] ? kNever : c[v];
        }
    }
    int key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = c[v] == kNever ? kNeverKey : key_of(c[v]);
    for (int k = 0; k < a.topk; ++k) {
        int m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
        const int best = lanes_max<L>(m);
        // the lowest of this token's lanes that holds it
        const uint64_t hold = __ballot(m == best);
        int holder;
        if constexpr (L == 64) {
            holder = (int)__builtin_ctzll(hold);
        } else {
            const uint32_t half = threadIdx.x & 32 ? (uint32_t)(hold >> 32) : (uint32_t)hold;
            holder = (int)__builtin_ctz(L == 32 ? half : half >> (threadIdx.x & 16));
        }
        if (holder == q) {
            int at = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) at = key[v] == best ? v : at;
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = v == at ? kNeverKey : key[v];
            chosen[g][k] = best == kNeverKey ? -1 : e0 + at;
        }
    }
    wave_sync();
    float total = 0.0f;
    for (int k = q; k < a.topk; k += L) {
        const int e = chosen[g][k];
        total += e >= 0 ? scores[g][e] / sum : 0.0f;
    }
    total = lanes_sum<L>(total);
    if (!live) return;
    for (int k = q; k < a.topk; k += L) {
        const int e = chosen[g][k];
        float w = e >= 0 ? scores[g][e] / sum : 0.0f;
        if (a.renorm && total > 0.0f) w = w / total;
        a.ids[t * a.topk + k] = e;
        a.weights[t * a.topk + k] = w * a.scale;
    }
}

// ------------------------------------------------------------------ dispatch

// A stable counting sort of the entries by expert.  Up to 4096 entries: one workgroup counts, scans
// and places (4096 entries 7.2 us; 6.5 in two launches, of which the second costs the host 3 us).  More: one launch counts each chunk's experts, a second places every chunk from
// the counts of the chunks before it; beyond 64 chunks a launch between them sums the counts over the
// chunks, so that no workgroup reads them all.  Within a chunk a wave takes consecutive entries, 64
// at a time; an entry's place among its wave's entries of the same expert comes from ballots over
// the expert's bits, so the order needs no atomics.  Bound: launches and dependent loads: 64 entries
// 4.0 us, 65536 entries of 128 experts (0.8 MB) 7.9 us, 2M entries of 256 experts (25 MB) 29 us.

constexpr int kDispThreads = 1024, kDispWaves = 16;
constexpr int kDispOnePer = 4;   // entries a thread of a call of one chunk (4096 entries)
constexpr int kDispDirect = 64;  // chunks whose counts a placing workgroup adds up itself

struct DispatchArgs {
    const int32_t* ids;
    int32_t *sorted_tok, *row_idx, *expert_off, *group_expert, *group_off;
    int32_t* counts;  // [chunk][expert]; summed: entries of the expert in the chunks before
    int32_t* totals;  // [expert], summed only
    int n, topk, nexperts, ngroups, chunks, bits;
};

__device__ __forceinline__ int expert_at(const DispatchArgs& a, int p) {
    const int e = p < a.n ? a.ids[p] : -1;
    return e >= 0 && e < a.nexperts ? e : -1;
}

// Inclusive scan over the workgroup (16 waves), the waves' sums through LDS.
__device__ __forceinline__ int workgroup_scan(int v, int* part) {
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    v = wave_scan(v);
    if (l == 63) part[w] = v;
    __syncthreads();
    for (int u = 0; u < w; ++u) v += part[u];
    return v;
}

// counts[chunk][e], chunks of 1024 PER entries
template <int PER>
__global__ __launch_bounds__(kDispThreads) void dispatch_count_kernel(DispatchArgs a) {
    __shared__ int count[kRouteMaxExperts];
    const int i = threadIdx.x, p0 = (int)blockIdx.x * (PER * kDispThreads);
    int e[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) e[u] = expert_at(a, p0 + u * kDispThreads + i);
    count[i] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (e[u] >= 0) atomicAdd(&count[e[u]], 1);
    __syncthreads();
    if (i < a.nexperts) a.counts[(int64_t)blockIdx.x * a.nexperts + i] = count[i];
}

// Workgroup of 64 experts: 16 runs of chunks each, counts replaced by the entries before the chunk.
__global__ __launch_bounds__(kDispThreads) void dispatch_sum_kernel(DispatchArgs a) {
    __shared__ int part[kDispWaves][64];
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6, e = (int)blockIdx.x * 64 + l;
    const int per = (a.chunks + kDispWaves - 1) / kDispWaves;
    const int c0 = w * per, c1 = c0 + per < a.chunks ? c0 + per : a.chunks;
    int s = 0;
    if (e < a.nexperts)
        for (int c = c0; c < c1; ++c) s += a.counts[(int64_t)c * a.nexperts + e];
    part[w][l] = s;
    __syncthreads();
    int before = 0;
    for (int u = 0; u < w; ++u) before += part[u][l];
    if (e >= a.nexperts) return;
    for (int c = c0; c < c1; ++c) {
        int32_t* p = a.counts + (int64_t)c * a.nexperts + e;
        const int v = *p;
        *p = before;
        before += v;
    }
    if (w == kDispWaves - 1) a.totals[e] = before;
}

enum { kDispOne, kDispAdd, kDispSummed };

// Workgroup = chunk of 1024 PER entries (kDispOne: all of them).  MODE: how the entries of the other
// chunks are known.
template <int MODE, int PER>
__global__ __launch_bounds__(kDispThreads) void dispatch_place_kernel(DispatchArgs a) {
    extern __shared__ uint16_t seen[];  // [wave][expert]: entries of the waves before, then of the wave so far
    __shared__ int first[kRouteMaxExperts], part[kDispWaves], every;
    const int i = threadIdx.x, l = i & 63, w = i >> 6, E = a.nexperts;
    // entries per wave: whole runs of 64, as even as they go
    const int per = MODE == kDispOne ? (a.n + kDispThreads - 1) / kDispThreads : PER;
    const int begin = (int)blockIdx.x * (PER * kDispThreads), p0 = begin + w * per * 64 + l;
    int e[PER], place[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) e[u] = u < per ? expert_at(a, p0 + 64 * u) : -1;

    int total = 0, before = 0;  // of expert i: all its entries, and those of earlier chunks
    if (i < E) {
        if constexpr (MODE == kDispAdd) {
#pragma unroll 8
            for (int c = 0; c < a.chunks; ++c) {
                const int v = a.counts[(int64_t)c * E + i];
                total += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
        } else if constexpr (MODE == kDispSummed) {
            total = a.totals[i];
            before = a.counts[(int64_t)blockIdx.x * E + i];
        }
    }
    uint16_t* mine = seen + w * E;
    for (int k = l; k < E; k += 64) mine[k] = 0;
    wave_sync();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        if (u >= per) break;
        uint64_t same = __ballot(e[u] >= 0);
        for (int b = 0; b < a.bits; ++b) {
            const uint64_t m = __ballot((e[u] >> b) & 1);
            same &= (e[u] >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << l) - 1ull));
        place[u] = e[u] >= 0 ? mine[e[u]] + rank : 0;
        wave_sync();
        if (e[u] >= 0 && rank == 0) mine[e[u]] = (uint16_t)(place[u] + __popcll(same));
        wave_sync();
    }
    __syncthreads();
    if (i < E) {
        int run = 0;
        for (int u = 0; u < kDispWaves; ++u) {
            const int v = seen[u * E + i];
            seen[u * E + i] = (uint16_t)run;
            run += v;
        }
        if constexpr (MODE == kDispOne) total = run;
    }
    const int end = workgroup_scan(total, part);
    if (i < E) first[i] = end - total + before;
    if (i == kDispThreads - 1) every = end;  // all entries
    __syncthreads();
    const int all = every;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int p = p0 + 64 * u;
        if (u >= per || p >= a.n) continue;
        const int at = e[u] >= 0 ? first[e[u]] + mine[e[u]] + place[u] : -1;
        a.row_idx[p] = at;
        if (at >= 0) a.sorted_tok[at] = p / a.topk;
    }
    for (int u = 0; u < PER; ++u) {
        const int p = begin + u * kDispThreads + i;
        if (p >= all && p < a.n) a.sorted_tok[p] = -1;
    }
    if (blockIdx.x == 0) {
        if (i < E) a.expert_off[i] = end - total;
        if (i == 0) a.expert_off[E] = all;
        if (a.group_off) {
            const int live = workgroup_scan(total > 0, part);
            if (total > 0) {
                a.group_expert[live - 1] = i;
                a.group_off[live - 1] = end - total;
            }
            if (i == kDispThreads - 1) every = live;
            __syncthreads();
            for (int g = every + i; g <= a.ngroups; g += kDispThreads) {
                if (g < a.ngroups) a.group_expert[g] = -1;
                a.group_off[g] = all;
            }
        }
    }
}

}  // namespace qmm

#include "qmm_types.h"

using namespace qmm;

constexpr int64_t kRouteMaxTokens = (1 << 25) - 1;  // 64 lanes a token, below 2^32 threads

extern "C" int qmm_moe_route(int ltype, const void* logits, int64_t ldl, const float* bias, int64_t ntok, int nexperts, int score,
                             int ngroups, int topk_groups, int group_top, int topk, float scale, int32_t* ids, float* weights,
                             unsigned flags, void* stream) {
    if (!valid_type(ltype) || (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) || (flags & ~QMM_ROUTE_RENORM))
        return QMM_EINVAL;
    if (ntok < 0 || nexperts < 1 || ldl < nexperts || ngroups < 1 || topk_groups < 1 || topk_groups > ngroups || topk < 1)
        return QMM_EINVAL;
    if (nexperts > kRouteMaxExperts || ngroups > kRouteMaxGroups || topk > kRouteMaxTopk || ntok > kRouteMaxTokens) return QMM_EUNSUPPORTED;
    if (nexperts % ngroups || topk > topk_groups * (nexperts / ngroups)) return QMM_EINVAL;
    if (group_top < 1 || group_top > 2 || group_top > nexperts / ngroups) return QMM_EINVAL;
    if (ntok == 0) return QMM_OK;
    if (!logits || !ids || !weights) return QMM_EINVAL;
    if (!aligned(logits, type_bytes(ltype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return QMM_EALIGN;
    const RouteArgs a{logits, bias, ldl, ntok, ltype, nexperts, score == QMM_SCORE_SOFTMAX, ngroups, topk_groups, group_top, topk,
                      (flags & QMM_ROUTE_RENORM) != 0, scale, ids, weights};
    const bool vec = nexperts % 8 == 0 && aligned(logits, 16) && ldl * (int64_t)type_bytes(ltype) % 16 == 0;
    const hipStream_t st = as_stream(stream);
    const auto grid = [&](int lanes) { return dim3((unsigned)((ntok * lanes + 255) / 256)); };
    const dim3 block(256);
    if (nexperts <= 32) hipLaunchKernelGGL((route_kernel<16, 2, false>), grid(16), block, 0, st, a);
    else if (nexperts <= 64) hipLaunchKernelGGL((route_kernel<16, 4, false>), grid(16), block, 0, st, a);
    else if (nexperts <= 128 && vec) hipLaunchKernelGGL((route_kernel<16, 8, true>), grid(16), block, 0, st, a);
    else if (nexperts <= 128) hipLaunchKernelGGL((route_kernel<16, 8, false>), grid(16), block, 0, st, a);
    else if (nexperts <= 256 && vec) hipLaunchKernelGGL((route_kernel<32, 8, true>), grid(32), block, 0, st, a);
    else if (nexperts <= 256) hipLaunchKernelGGL((route_kernel<32, 8, false>), grid(32), block, 0, st, a);
    else if (nexperts <= 512 && vec) hipLaunchKernelGGL((route_kernel<64, 8, true>), grid(64), block, 0, st, a);
    else if (nexperts <= 512) hipLaunchKernelGGL((route_kernel<64, 8, false>), grid(64), block, 0, st, a);
    else if (vec) hipLaunchKernelGGL((route_kernel<64, 16, true>), grid(64), block, 0, st, a);
    else hipLaunchKernelGGL((route_kernel<64, 16, false>), grid(64), block, 0, st, a);
    return launch_status();
}

// Entries a thread of a chunked call: 2 while a placing workgroup can add up all counts (65536 entries
// 8.0 us; 9.2 with 4), else 8 (2M entries 29 us; 46 with 2).
static int dispatch_per(int64_t n) { return n <= kDispDirect * 2 * kDispThreads ? 2 : 8; }
static int64_t dispatch_chunks(int64_t n) {
    const int64_t chunk = dispatch_per(n) * kDispThreads;
    return n <= kDispOnePer * kDispThreads ? 1 : (n + chunk - 1) / chunk;
}

static bool dispatch_takes(int64_t ntok, int topk, int nexperts) {
    return ntok <= 0x7FFFFFFF && topk <= kRouteMaxTopk && nexperts <= kRouteMaxExperts && ntok * topk <= (int64_t)1 << 30;
}

extern "C" size_t qmm_moe_dispatch_workspace(int64_t ntok, int topk, int nexperts) {
    if (ntok < 0 || topk < 1 || nexperts < 1 || !dispatch_takes(ntok, topk, nexperts)) return 0;
    const int64_t chunks = dispatch_chunks(ntok * topk);
    return chunks == 1 ? 16 : (size_t)(chunks + 1) * nexperts * 4;
}

extern "C" int qmm_moe_dispatch(const int32_t* ids, int64_t ntok, int topk, int nexperts, int32_t* sorted_tok, int32_t* row_idx,
                                int32_t* expert_off, int32_t* group_expert, int32_t* group_off, void* ws, size_t ws_bytes,
                                void* stream) {
    if (ntok < 0 || topk < 1 || nexperts < 1 || !expert_off || (group_expert && !group_off)) return QMM_EINVAL;
    if (!dispatch_takes(ntok, topk, nexperts)) return QMM_EUNSUPPORTED;
    if (ntok && (!ids || !sorted_tok || !row_idx || !ws || (group_off && !group_expert))) return QMM_EINVAL;
    if (!aligned(ids, 4) || !aligned(sorted_tok, 4) || !aligned(row_idx, 4) || !aligned(expert_off, 4) || !aligned(group_expert, 4) ||
        !aligned(group_off, 4) || !aligned(ws, 4))
        return QMM_EALIGN;
    if (ntok && ws_bytes < qmm_moe_dispatch_workspace(ntok, topk, nexperts)) return QMM_ESPACE;
    const int n = (int)(ntok * topk);
    const int chunks = (int)dispatch_chunks(n);
    int bits = 0;
    while ((1 << bits) < nexperts) ++bits;
    int32_t* const counts = (int32_t*)ws;
    const DispatchArgs a{ids, sorted_tok, row_idx, expert_off, group_expert, group_off, counts, counts + (int64_t)chunks * nexperts,
                         n, topk, nexperts, n < nexperts ? n : nexperts, chunks, bits};
    const hipStream_t st = as_stream(stream);
    const size_t lds = (size_t)kDispWaves * nexperts * 2;
    const dim3 block(kDispThreads);
    if (chunks == 1) {
        hipLaunchKernelGGL((dispatch_place_kernel<kDispOne, kDispOnePer>), dim3(1), block, lds, st, a);
    } else if (dispatch_per(n) == 2) {
        hipLaunchKernelGGL(dispatch_count_kernel<2>, dim3((unsigned)chunks), block, 0, st, a);
        hipLaunchKernelGGL((dispatch_place_kernel<kDispAdd, 2>), dim3((unsigned)chunks), block, lds, st, a);
    } else if (chunks <= kDispDirect) {
        hipLaunchKernelGGL(dispatch_count_kernel<8>, dim3((unsigned)chunks), block, 0, st, a);
        hipLaunchKernelGGL((dispatch_place_kernel<kDispAdd, 8>), dim3((unsigned)chunks), block, lds, st, a);
    } else {
        hipLaunchKernelGGL(dispatch_count_kernel<8>, dim3((unsigned)chunks), block, 0, st, a);
        hipLaunchKernelGGL(dispatch_sum_kernel, dim3((unsigned)((nexperts + 63) / 64)), block, 0, st, a);
        hipLaunchKernelGGL((dispatch_place_kernel<kDispSummed, 8>), dim3((unsigned)chunks), block, lds, st, a);
    }
    return launch_status();
}
