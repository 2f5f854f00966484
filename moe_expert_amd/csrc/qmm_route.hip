// qmm_route.hip -- routing of tokens to experts and the expert-sorted entry lists, for gfx950.
#include "qmm_values.h"

namespace qmm {

constexpr int kRouteMaxExperts = 1024, kRouteMaxTopk = 64, kRouteMaxGroups = 64;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t ldl;
    int ltype, nexperts, softmax, ngroups, topk_groups, group_top, topk, renorm;
    float scale;
    int32_t* ids;
    float* weights;
};

__device__ __forceinline__ float wave_max(float v) {
    for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

constexpr float kNever = -__builtin_inff();

// One wave per token.  score[e] and choice[e] in LDS (choice -inf: never chosen); the best of the
// choices is taken topk times, ties to the lowest index.
__global__ __launch_bounds__(64) void route_kernel(RouteArgs a) {
    __shared__ float score[kRouteMaxExperts], choice[kRouteMaxExperts], run[kRouteMaxGroups], wsel[kRouteMaxTopk];
    const int64_t t = blockIdx.x;
    const int l = threadIdx.x, E = a.nexperts;
    float top = kNever;
    for (int e = l; e < E; e += 64) {
        const float z = load_value(a.logits, t * a.ldl + e, a.ltype);
        choice[e] = z == z ? z : kNever;
        top = fmaxf(top, choice[e]);
    }
    top = wave_max(top);
    float sum = 0.0f;
    if (a.softmax) {
        for (int e = l; e < E; e += 64) {
            const float z = choice[e];
            score[e] = z == kNever ? 0.0f : z == top ? 1.0f : expf(z - top);
            sum += score[e];
        }
        sum = wave_sum(sum);
    }
    const bool by_logit = a.softmax && !a.bias && (a.ngroups == 1 || a.group_top == 1);
    for (int e = l; e < E; e += 64) {
        const float z = choice[e];
        const float s = a.softmax ? (sum > 0.0f ? score[e] / sum : 0.0f) : 1.0f / (1.0f + expf(-z));
        score[e] = s;
        if (!by_logit && z != kNever) {
            const float c = a.bias ? s + a.bias[e] : s;
            choice[e] = c == c ? c : kNever;
        }
    }
    __syncthreads();
    if (a.ngroups > 1) {
        const int per = E / a.ngroups;
        if (l < a.ngroups) {
            float m0 = kNever, m1 = kNever;
            for (int i = 0; i < per; ++i) {
                const float c = choice[l * per + i];
                if (c > m0) { m1 = m0; m0 = c; }
                else if (c > m1) m1 = c;
            }
            run[l] = a.group_top == 2 ? (m1 == kNever ? kNever : m0 + m1) : m0;
        }
        __syncthreads();
        if (l < a.ngroups) {
            int better = 0;
            for (int g = 0; g < a.ngroups; ++g) better += run[g] > run[l] || (run[g] == run[l] && g < l);
            if (better >= a.topk_groups)
                for (int i = 0; i < per; ++i) choice[l * per + i] = kNever;
        }
        __syncthreads();
    }
    float total = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
        float best = kNever;
        int at = E;
        for (int e = l; e < E; e += 64)
            if (choice[e] > best) { best = choice[e]; at = e; }
        const float m = wave_max(best);
        if (best != m || m == kNever) at = E;
        for (int d = 32; d; d >>= 1) {
            const int o = __shfl_xor(at, d, 64);
            at = o < at ? o : at;
        }
        const bool found = at < E;
        const float s = found ? score[at] : 0.0f;
        total += s;
        __syncthreads();
        if (l == 0) {
            if (found) choice[at] = kNever;
            a.ids[t * a.topk + k] = found ? at : -1;
            wsel[k] = s;
        }
        __syncthreads();
    }
    if (l < a.topk) {
        float w = wsel[l];
        if (a.renorm && total > 0.0f) w = w / total;
        a.weights[t * a.topk + l] = w * a.scale;
    }
}

// ------------------------------------------------------------------ dispatch

struct DispatchArgs {
    const int32_t* ids;
    int n, topk, nexperts, ngroups;
    int32_t *sorted_tok, *row_idx, *expert_off, *group_expert, *group_off;
};

constexpr int kDispThreads = 1024;

// One workgroup: counts per expert, their prefix sums, then the entries in order, 64 at a time by
// one wave, so that each expert's entries keep their order.
__global__ __launch_bounds__(kDispThreads) void dispatch_kernel(DispatchArgs a) {
    __shared__ int count[kRouteMaxExperts], scan[kDispThreads], live[kDispThreads];
    const int i = threadIdx.x;
    count[i] = 0;
    __syncthreads();
    for (int p = i; p < a.n; p += kDispThreads) {
        const int e = a.ids[p];
        if (e >= 0 && e < a.nexperts) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    const int c = count[i];
    scan[i] = c;
    live[i] = c > 0;
    __syncthreads();
    for (int d = 1; d < kDispThreads; d <<= 1) {
        const int u = i >= d ? scan[i - d] : 0, v = i >= d ? live[i - d] : 0;
        __syncthreads();
        scan[i] += u;
        live[i] += v;
        __syncthreads();
    }
    const int total = scan[kDispThreads - 1], nlive = live[kDispThreads - 1], first = scan[i] - c;
    if (i < a.nexperts) a.expert_off[i] = first;
    if (i == 0) a.expert_off[a.nexperts] = total;
    if (a.group_off) {
        if (c > 0) {
            a.group_expert[live[i] - 1] = i;
            a.group_off[live[i] - 1] = first;
        }
        for (int g = nlive + i; g <= a.ngroups; g += kDispThreads) {
            if (g < a.ngroups) a.group_expert[g] = -1;
            a.group_off[g] = total;
        }
    }
    for (int p = total + i; p < a.n; p += kDispThreads) a.sorted_tok[p] = -1;
    __syncthreads();
    count[i] = first;
    __syncthreads();
    if (i < 64) {
        for (int p0 = 0; p0 < a.n; p0 += 64) {
            const int p = p0 + i;
            int e = p < a.n ? a.ids[p] : -1;
            if (e < 0 || e >= a.nexperts) e = -1;
            unsigned long long same = ~0ull;
            for (int b = 0; b < 11; ++b) {
                const unsigned long long m = __ballot((e >> b) & 1);
                same &= ((e >> b) & 1) ? m : ~m;
            }
            const int rank = __popcll(same & ((1ull << i) - 1ull));
            const int at = e >= 0 ? count[e] + rank : -1;
            __builtin_amdgcn_wave_barrier();
            if (e >= 0 && rank == 0) count[e] += __popcll(same);
            __builtin_amdgcn_wave_barrier();
            if (p < a.n) a.row_idx[p] = at;
            if (at >= 0) a.sorted_tok[at] = p / a.topk;
        }
    }
}

}  // namespace qmm

#include "qmm_host.h"

using namespace qmm;

extern "C" int qmm_moe_route(int ltype, const void* logits, int64_t ldl, const float* bias, int64_t ntok, int nexperts, int score,
                             int ngroups, int topk_groups, int group_top, int topk, float scale, int32_t* ids, float* weights,
                             unsigned flags, void* stream) {
    if (!valid_type(ltype) || (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) || (flags & ~QMM_ROUTE_RENORM))
        return QMM_EINVAL;
    if (ntok < 0 || nexperts < 1 || ldl < nexperts || ngroups < 1 || topk_groups < 1 || topk_groups > ngroups || topk < 1)
        return QMM_EINVAL;
    if (nexperts > kRouteMaxExperts || ngroups > kRouteMaxGroups || topk > kRouteMaxTopk || ntok > 0x7FFFFFFF) return QMM_EUNSUPPORTED;
    if (nexperts % ngroups || topk > topk_groups * (nexperts / ngroups)) return QMM_EINVAL;
    if (group_top < 1 || group_top > 2 || group_top > nexperts / ngroups) return QMM_EINVAL;
    if (ntok == 0) return QMM_OK;
    if (!logits || !ids || !weights) return QMM_EINVAL;
    if (!aligned(logits, type_bytes(ltype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return QMM_EALIGN;
    RouteArgs a{logits, bias, ldl, ltype, nexperts, score == QMM_SCORE_SOFTMAX, ngroups, topk_groups, group_top, topk,
                (flags & QMM_ROUTE_RENORM) != 0, scale, ids, weights};
    hipLaunchKernelGGL(route_kernel, dim3((unsigned)ntok), dim3(64), 0, as_stream(stream), a);
    return launch_status();
}

static bool dispatch_takes(int64_t ntok, int topk, int nexperts) {
    return ntok <= 0x7FFFFFFF && topk <= kRouteMaxTopk && nexperts <= kRouteMaxExperts && ntok * topk <= 0x7FFFFFFF;
}

extern "C" size_t qmm_moe_dispatch_workspace(int64_t ntok, int topk, int nexperts) {
    if (ntok < 0 || topk < 1 || nexperts < 1 || !dispatch_takes(ntok, topk, nexperts)) return 0;
    return 16;
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
    DispatchArgs a{ids, n, topk, nexperts, n < nexperts ? n : nexperts, sorted_tok, row_idx, expert_off, group_expert, group_off};
    hipLaunchKernelGGL(dispatch_kernel, dim3(1), dim3(kDispThreads), 0, as_stream(stream), a);
    return launch_status();
}
