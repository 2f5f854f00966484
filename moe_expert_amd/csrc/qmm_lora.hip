// qmm_lora.hip -- low-rank adapters of many requests beside a shared projection, for gfx950:
// y[t] = base[t] + scale_i * B_i (A_i x[t]), i the adapter of the token's segment.
//
// Two launches, each over tiles of the tokens of one segment (found by a scan of the segments, so
// their lengths stay on the device): the inner values v = A_i x[t] in binary32 into the workspace,
// then the outer product added to the base.  (Both in one launch, each workgroup forming the inner
// values for itself, measured slower: 9.4 against 8.0 us for 8 requests of one token at rank 16,
// k 2560, 8192 rows; 40 against 13 us at rank 64, k 6144, 2560 rows.)
//
// Bound: the base and y.  8192 tokens x (2560 -> 8192), rank 16: 130 us for the 580 MB that cannot be
// avoided (4.5 TB/s, a large copy reaches 5.0), of which the inner values 18 us; short calls are
// bound by the chain of dependent loads segment -> adapter -> A, x -> inner values -> y.  Many requests
// of one token are far from their bytes (64: 14.7 us for 9 MB; 512, 2560 -> 2560: 42 us; 4096,
// 1024 -> 1024: 209 us): a tile of 32 tokens each, found by a scan of the segments in each workgroup.
#include "qmm_values.h"

namespace qmm {

constexpr int kLoraMaxRank = 256;

struct LoraArgs {
    const void* x;
    const uint16_t *a, *b;
    const int32_t *ranks, *seg_off, *seg_adapter;
    const float *scales, *base;
    float *y, *v;
    int64_t ldx, ldbase, ldy;
    int ntok, k, nadapters, max_rank, nseg, nrows, split;
};

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct LoraTile {
    int t0, nt, adapter, rank;  // nt = 0: no such tile
    float scale;
};

// Tile `tile` of the segments' tiles of T tokens each (the last of a segment holds what is left):
// its tokens [t0, t0 + nt) and their adapter, -1 for none.  A scan of the segments' tile counts, 64 a
// step; MANY, for more than 64 segments: four steps are skipped by their sum where the tile lies
// beyond them (4096 segments 223 us against 407 when it was tried).  Every wave does its own, all lanes call it.
template <bool MANY>
__device__ __forceinline__ LoraTile find_tile(const LoraArgs& a, int T, int tile) {
    const int l = threadIdx.x & 63;
    for (int s0 = 0; s0 < a.nseg; s0 += 64) {
        if constexpr (MANY) {
            while (s0 + 256 <= a.nseg) {
                int total = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    int o0 = a.seg_off[s0 + 64 * u + l], o1 = a.seg_off[s0 + 64 * u + l + 1];
                    o0 = o0 < 0 ? 0 : o0 > a.ntok ? a.ntok : o0;
                    o1 = o1 < o0 ? o0 : o1 > a.ntok ? a.ntok : o1;
                    total += (o1 - o0 + T - 1) / T;
                }
                total = __builtin_amdgcn_readlane(wave_scan(total), 63);
                if (total > tile) break;
                tile -= total;
                s0 += 256;
            }
        }
        const int s = s0 + l;
        int o0 = 0, o1 = 0, i = -1;
        if (s < a.nseg) {
            o0 = a.seg_off[s];
            o1 = a.seg_off[s + 1];
            i = a.seg_adapter[s];
        }
        int rank = 0;
        float scale = 0.0f;
        if (i >= 0 && i < a.nadapters) {  // on their way during the scan
            rank = a.ranks[i];
            scale = a.scales[i];
        } else {
            i = -1;
        }
        o0 = o0 < 0 ? 0 : o0 > a.ntok ? a.ntok : o0;
        o1 = o1 < o0 ? o0 : o1 > a.ntok ? a.ntok : o1;
        const int n = (o1 - o0 + T - 1) / T;
        const int upto = wave_scan(n);
        const uint64_t past = __ballot(upto > tile);
        if (past) {
            const int src = (int)__builtin_ctzll(past);
            LoraTile r;
            r.t0 = __builtin_amdgcn_readlane(o0, src) + (tile - __builtin_amdgcn_readlane(upto - n, src)) * T;
            const int left = __builtin_amdgcn_readlane(o1, src) - r.t0;
            r.nt = left < T ? left : T;
            r.adapter = __builtin_amdgcn_readlane(i, src);
            r.rank = __builtin_amdgcn_readlane(rank, src);
            r.rank = r.rank < 0 ? 0 : r.rank > a.max_rank ? a.max_rank : r.rank;
            r.scale = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scale), src));
            return r;
        }
        tile -= __builtin_amdgcn_readlane(upto, 63);
    }
    return {0, 0, -1, 0, 0.0f};
}

// ------------------------------------------------------------------ inner values

// One step of 32 columns: 8 values of x of a token row, 8 values of A of each of NR blocks of 16
// rank rows; lane l holds row l % 16 and columns 8 (l / 16) .. + 7 of the step.
template <int XT, int NR>
struct DownStep {
    u32x4 x[XT == kF32 ? 2 : 1];
    u32x4 a[NR];
};

// The inner values of a tile of up to 16 tokens into part[wave][token][rank row], each wave the
// sum over its run of 32-column steps (wave `run` of `runs`).  Rows past the tile or the rank read
// the last valid row; what they give is not used.
template <int XT, int NR, int LD>
__device__ __forceinline__ void down_tile(const LoraArgs& a, const LoraTile& tile, int run, int runs, float (*part)[LD]) {
    constexpr int U = NR <= 2 ? 8 : NR <= 4 ? 4 : 2;  // steps whose loads are in flight together
    const int l = threadIdx.x & 63, row = l & 15, q = l >> 4;
    const char* xr = (const char*)a.x + ((int64_t)(tile.t0 + (row < tile.nt ? row : tile.nt - 1)) * a.ldx + 8 * q) * (XT == kF32 ? 4 : 2);
    const uint16_t* ar[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int j = 16 * n + row;
        ar[n] = a.a + ((int64_t)tile.adapter * a.max_rank + (j < tile.rank ? j : tile.rank - 1)) * a.k + 8 * q;
    }
    const int steps = a.k / 32;
    const int per = (steps + runs - 1) / runs;
    const int c0 = run * per, c1 = c0 + per < steps ? c0 + per : steps;

    f32x4 acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4{};

    auto load = [&](DownStep<XT, NR>& s, int c) {
        const u32x4* p = (const u32x4*)(xr + (int64_t)c * (XT == kF32 ? 128 : 64));
        s.x[0] = p[0];
        if constexpr (XT == kF32) s.x[1] = p[1];
#pragma unroll
        for (int n = 0; n < NR; ++n) s.a[n] = *(const u32x4*)(ar[n] + (int64_t)c * 32);
    };
    auto apply = [&](const DownStep<XT, NR>& s) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const half8 b = __builtin_bit_cast(half8, s.a[n]);
            if constexpr (XT == kF32) {
                const f32x4 x0 = __builtin_bit_cast(f32x4, s.x[0]), x1 = __builtin_bit_cast(f32x4, s.x[1]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(e < 4 ? x0[e] : x1[e - 4], (float)b[e], acc[n], 0, 0, 0);
            } else {
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, s.x[0]), b, acc[n], 0, 0, 0);
            }
        }
    };
    for (int c = c0; c < c1; c += U) {
        DownStep<XT, NR> s[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u < c1) load(s[u], c + u);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u < c1) apply(s[u]);
    }
    // accumulator register r of lane l: token 4 (l / 16) + r, rank row l % 16
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[4 * q + r][16 * n + row] = acc[n][r];
}

// The same for the blocks of 16 rank rows that the adapter uses, 1, 2, 4, ... up to the table's NR.
template <int XT, int NR, int LD>
__device__ __forceinline__ void down_tile_ranks(const LoraArgs& a, const LoraTile& tile, int run, int runs, float (*part)[LD]) {
    if constexpr (NR > 1) {
        if (tile.rank <= 8 * NR) return down_tile_ranks<XT, NR / 2, LD>(a, tile, run, runs, part);
    }
    down_tile<XT, NR, LD>(a, tile, run, runs, part);
}

// Workgroup (tile, split): the waves' sums joined in wave order into the split's inner values.  16
// tokens a tile (32 measured the same on prompts and leave half as many workgroups in short calls);
// 8192 tokens, k 2560, rank 16: 17.6 us for the 42 MB of x; 517 tokens, ranks to 64: 9.3 us.
template <int XT, int NR, int W, bool MANY>
__global__ __launch_bounds__(64 * W) void lora_down_kernel(LoraArgs a) {
    constexpr int T = 16, R = 16 * NR;
    __shared__ float part[W][T][R + 1];
    const LoraTile tile = find_tile<MANY>(a, T, blockIdx.x);
    if (tile.nt == 0 || tile.rank == 0) return;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    down_tile_ranks<XT, NR, R + 1>(a, tile, (int)blockIdx.y * W + w, W * a.split, part[w]);
    __syncthreads();
    float* v = a.v + ((int64_t)blockIdx.y * a.ntok + tile.t0) * a.max_rank;
    for (int i = threadIdx.x; i < tile.nt * R; i += 64 * W) {
        const int t = i / R, j = i % R;
        if (j >= ((tile.rank + 7) & ~7)) continue;  // the outer product reads whole groups of 8
        float s = part[0][t][j];
#pragma unroll
        for (int u = 1; u < W; ++u) s += part[u][t][j];
        v[(int64_t)t * a.max_rank + j] = j < tile.rank ? s : 0.0f;
    }
}

// ------------------------------------------------------------------ outer product

constexpr int kUpTokens = 32, kUpRows = 256;  // of y per workgroup: one block of 64 rows a wave

// A binary32 value as three bfloat16 parts, v = v1 + v2 + v3 exactly (8 bits each, cut, not rounded, so
// none overflows); an infinity or NaN is the first part alone.  Parts are the high halves of words.
__device__ __forceinline__ void split3(float v, uint32_t* p) {
    p[0] = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
    p[1] = p[2] = 0;
    if (v != v) p[0] = 0x7FC00000u;
    if (__builtin_isfinite(v)) {
        const float r = v - __builtin_bit_cast(float, p[0]);
        p[1] = __builtin_bit_cast(uint32_t, r) & 0xFFFF0000u;
        p[2] = __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, p[1]));
    }
}

// The high halves of two words as one.
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// The inner values of a tile in LDS, each as its three parts, in the order the outer product's A operand
// takes them.  frag: [part][step of 16 ranks][half][token], 8 consecutive ranks each; zeros past the
// rank and past the tile's tokens.  fetch(token, j, v) adds the values j .. j+7 of a token to v.
template <class F>
__device__ __forceinline__ void make_fragments(const LoraTile& tile, u32x4* frag, F fetch) {
    constexpr int T = kUpTokens, G = 256 / T;  // G threads per token
    const int tok = threadIdx.x % T, steps = (tile.rank + 15) / 16, part = steps * 2 * T;
#pragma unroll 1
    for (int g = threadIdx.x / T; g < 2 * steps; g += G) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        if (tok < tile.nt && 8 * g < tile.rank) fetch(tok, 8 * g, v);
        uint32_t p[8][3];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3(8 * g + e < tile.rank ? v[e] : 0.0f, p[e]);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            u32x4 w;
            w.x = high_halves(p[0][n], p[1][n]);
            w.y = high_halves(p[2][n], p[3][n]);
            w.z = high_halves(p[4][n], p[5][n]);
            w.w = high_halves(p[6][n], p[7][n]);
            frag[n * part + g * T + tok] = w;
        }
    }
    __syncthreads();
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// A wave's block of y: the tile's 32 tokens by 64 rows (from row rb of the workgroup's).  Column l % 32
// of product c takes row 2 (l % 32) + c, so a lane holds two neighbouring values of each token:
// register r is token 8 (r / 4) + 4 (l / 32) + r % 4.  Every load is unconditional, at a clamped place
// where the block ends inside the tile or the rows (with a branch around each load the wave waited
// for one before the next: 8192 x 8192 took 190 us against 123).  y is stored past the caches (129 us
// against 144), the base is not read past them (517 tokens 23.2 us against 27.2): the projection has
// just written it.  The product is binary32's on bfloat16 MFMA: the three parts of a value times the two
// of B (11 bits), six exact products into the binary32 sum.  The binary32 MFMA instead has a sixteenth
// of the rate (517 tokens 25.2 us against 23.8; 64 requests of one token 18.5 against 14.6; 8192 tokens
// at rank 256 336 against 306).  FEW: tiles of up to 8 tokens skip the registers of the others.
// VEC: an even number of rows, aligned.
template <bool VEC, bool FEW>
struct UpBlock {
    static constexpr int CT = 2;
    f32x2 in[16];
    half8 b[2][CT];  // the next two 16-rank steps of B
    const uint16_t* br[CT];
    int j, h, col, rows;

    __device__ __forceinline__ UpBlock(int rb, int rows_) : rows(rows_) {
        const int l = threadIdx.x & 63;
        col = l & 31;
        h = l >> 5;
        j = rb + CT * col;
    }
    __device__ __forceinline__ int token(int r) const { return 8 * (r / 4) + 4 * h + r % 4; }
    // 16-rank step s of B, as it lies there
    __device__ __forceinline__ void load_b(half8* w, const LoraArgs& a, int s) const {
        const int k = 16 * s + 8 * h;
#pragma unroll
        for (int c = 0; c < CT; ++c) w[c] = *(const half8*)(br[c] + (k < a.max_rank ? k : 0));
    }
    __device__ __forceinline__ void load(const LoraArgs& a, const LoraTile& tile, int r0, const float* base) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (FEW && r == 4 && tile.nt <= 8) break;  // registers 4 and on are tokens 8 and on
            const int t = token(r);
            const float* p = base + (uint64_t)(uint32_t)(t < tile.nt ? t : tile.nt - 1) * (uint32_t)a.ldbase;
            if constexpr (VEC) {
                in[r] = *((const f32x2*)(p + (j < rows ? j : 0)));
            } else {
#pragma unroll
                for (int c = 0; c < CT; ++c) in[r][c] = p[j + c < rows ? j + c : rows - 1];
            }
        }
#pragma unroll
        for (int c = 0; c < CT; ++c)
            br[c] = a.b + ((int64_t)tile.adapter * a.nrows + r0 + (j + c < rows ? j + c : rows - 1)) * a.max_rank;
        load_b(b[0], a, 0);
        if (tile.rank > 16) load_b(b[1], a, 1);
    }
    // Columns of B past the rank may hold anything: zeros there.
    __device__ __forceinline__ void mask_b(half8& w, int s, int rank) const {
        if (16 * s + 16 > rank) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 16 * s + 8 * h + e < rank ? w[e] : (_Float16)0.0f;
        }
    }
    __device__ __forceinline__ void multiply_store(const LoraArgs& a, const LoraTile& tile, const u32x4* frag, float* y) {
        constexpr int T = kUpTokens;
        const int steps = (tile.rank + 15) / 16, part = steps * 2 * T;
        f32x16 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = f32x16{};
        for (int s = 0; s < steps; s += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (s + u >= steps) break;
                const u32x4* f = frag + (2 * (s + u) + h) * T + col;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    mask_b(b[u][c], s + u, tile.rank);
                    u32x4 w1, w2;  // w = w1 + w2 exactly: 8 and 3 bits
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float lo = (float)b[u][c][2 * i], hi = (float)b[u][c][2 * i + 1];
                        const uint32_t lu = __builtin_bit_cast(uint32_t, lo), hu = __builtin_bit_cast(uint32_t, hi);
                        w1[i] = high_halves(lu, hu);
                        w2[i] = high_halves(__builtin_bit_cast(uint32_t, lo - __builtin_bit_cast(float, lu & 0xFFFF0000u)),
                                            __builtin_bit_cast(uint32_t, hi - __builtin_bit_cast(float, hu & 0xFFFF0000u)));
                    }
#pragma unroll
                    for (int n = 2; n >= 0; --n) {
                        const bf8 v = __builtin_bit_cast(bf8, f[n * part]);
                        acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf8, w2), acc[c], 0, 0, 0);
                        acc[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf8, w1), acc[c], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // what is in flight across it did not fit the registers
                }
                if (s + u + 2 < steps) load_b(b[u], a, s + u + 2);
            }
        }
        // An infinity times the parts of a value is not the infinity times the value (a part may be 0 or of
        // the other sign): sums that are not finite are formed once more in binary32, the others stay.
        float odd = 0.0f;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) odd = __builtin_fmaf(acc[c][r], 0.0f, odd);
        uint32_t redo = 0;
        if (odd != odd) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!__builtin_isfinite(acc[c][r])) {
                        acc[c][r] = 0.0f;
                        redo |= 1u << (16 * c + r);
                    }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (FEW && r == 4 && tile.nt <= 8) break;
#pragma unroll
            for (int c = 0; c < CT; ++c) in[r][c] = in[r][c] + acc[c][r] * tile.scale;
        }
        if (__ballot(redo != 0)) add_in_binary32(a, tile, frag, redo);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (FEW && r == 4 && tile.nt <= 8) break;
            const int t = token(r);
            float* p = y + (uint64_t)(uint32_t)t * (uint32_t)a.ldy + j;
            if constexpr (VEC) {
                if (t < tile.nt && j < rows) __builtin_nontemporal_store(in[r], (f32x2*)p);
            } else if (t < tile.nt) {
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    if (j + c < rows) p[c] = in[r][c];
            }
        }
    }
    __device__ __forceinline__ void add_in_binary32(const LoraArgs& a, const LoraTile& tile, const u32x4* frag, uint32_t redo) {
        constexpr int T = kUpTokens;
        const int steps = (tile.rank + 15) / 16, part = steps * 2 * T;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            f32x16 sum = f32x16{};
#pragma unroll 1
            for (int s = 0; s < steps; ++s) {
                const u32x4* f = frag + (2 * s + h) * T + col;
                load_b(b[0], a, s);
                mask_b(b[0][c], s, tile.rank);
                const u32x4 v1 = f[0], v2 = f[part], v3 = f[2 * part];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const auto value = [&](const u32x4& p) {
                        return __builtin_bit_cast(float, e & 1 ? p[e / 2] & 0xFFFF0000u : p[e / 2] << 16);
                    };
                    sum = __builtin_amdgcn_mfma_f32_32x32x2f32(value(v1) + (value(v2) + value(v3)), (float)b[0][c][e], sum, 0, 0, 0);
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (redo >> (16 * c + r) & 1) in[r][c] += sum[r] * tile.scale;
        }
    }
};

// A workgroup's part of a tile without an adapter: y = base, one value a thread and token.  8192 x 8192
// without adapters: 202 us (537 MB, 2.7 TB/s).
__device__ __forceinline__ void copy_base(const LoraArgs& a, const LoraTile& tile, const float* base, float* y, int rows) {
    if (a.base == a.y) return;
    for (int t = 0; t < tile.nt; ++t)
        for (int j = threadIdx.x; j < rows; j += blockDim.x) y[t * a.ldy + j] = base[t * a.ldbase + j];
}

// Workgroup (row block, tile): 32 tokens by 256 rows of y, one UpBlock a wave, on the SPLIT parts of
// the inner values that lora_down_kernel left.  4 waves per SIMD (at 3 the prompt took 149 us against
// 138, at 5 the registers spill).  8192 x 8192, rank 16: 108 us for 537 MB; 517 x 12288, ranks to 64:
// 14.2 us for 63 MB.
template <int SPLIT, bool VEC, bool MANY, bool FEW>
__global__ __launch_bounds__(256, SPLIT > 2 ? 2 : 4) void lora_up_kernel(LoraArgs a) {
    constexpr int T = kUpTokens, ROWS = kUpRows;
    extern __shared__ u32x4 frag[];
    const LoraTile tile = find_tile<MANY>(a, T, blockIdx.y);
    if (tile.nt == 0) return;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r0 = (int)blockIdx.x * ROWS;
    const float* base = a.base + (int64_t)tile.t0 * a.ldbase + r0;
    float* y = a.y + (int64_t)tile.t0 * a.ldy + r0;
    const int rows = a.nrows - r0 < ROWS ? a.nrows - r0 : ROWS;
    if (tile.rank == 0) return copy_base(a, tile, base, y, rows);
    UpBlock<VEC, FEW> blk(64 * w, rows);
    blk.load(a, tile, r0, base);
    make_fragments(tile, frag, [&](int tok, int j, float* v) {
        const float* p = a.v + ((int64_t)tile.t0 + tok) * a.max_rank + j;
        f32x4 u[SPLIT][2];
#pragma unroll
        for (int s = 0; s < SPLIT; ++s) {
            const f32x4* ps = (const f32x4*)(p + (int64_t)s * a.ntok * a.max_rank);
            u[s][0] = ps[0];
            u[s][1] = ps[1];
        }
#pragma unroll
        for (int s = 0; s < SPLIT; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += u[s][e / 4][e % 4];
    });
    blk.multiply_store(a, tile, frag, y);
}

}  // namespace qmm

#include "qmm_types.h"

using namespace qmm;

constexpr int64_t kLoraMaxTokens = 1 << 20;
constexpr int kLoraMaxSegments = 1 << 14;

// How many workgroups share the columns of one token tile, so that few tiles still fill the GPU; the
// outer product reads that many parts.  With 1 / 2 / 8: 8 requests of one token at rank 16 10.9 / 8.6 /
// 7.3 us; one request (2560 -> 8192, rank 16) of 64 tokens 11.2 / 9.3 / 8.3, 256 tokens 13.2 / 11.2 / 10.3,
// 1024 tokens 20.2 / 18.2 / 19.7, 1100 tokens 21.0 / 19.2 / 20.3, 2048 tokens 29.6 / 28.9 / 31.9; 517
// ragged tokens, ranks to 64, 30.4 / 25.2 / 25.0.  The steps at 64 and 1024 tokens lie where the work per
// token still differs by 1 us (65 tokens 9.4 against 8.4) and 2 us (1100 tokens 21.1 against 19.2).
static int lora_split(int64_t ntok) { return ntok <= 64 ? 8 : ntok <= 1024 ? 2 : 1; }

extern "C" size_t qmm_lora_workspace(int64_t ntok, int max_rank) {
    if (ntok < 0 || ntok > kLoraMaxTokens || max_rank < 8 || max_rank % 8 || max_rank > kLoraMaxRank) return 0;
    return (size_t)lora_split(ntok) * ntok * max_rank * 4 + 16;
}

template <int XT, bool MANY>
static void launch_down(const LoraArgs& p, hipStream_t st) {
    const dim3 grid((unsigned)(p.ntok / 16 + p.nseg), (unsigned)p.split);
    if (p.max_rank <= 16) hipLaunchKernelGGL((lora_down_kernel<XT, 1, 8, MANY>), grid, dim3(512), 0, st, p);
    else if (p.max_rank <= 32) hipLaunchKernelGGL((lora_down_kernel<XT, 2, 8, MANY>), grid, dim3(512), 0, st, p);
    else if (p.max_rank <= 64) hipLaunchKernelGGL((lora_down_kernel<XT, 4, 8, MANY>), grid, dim3(512), 0, st, p);
    else if (p.max_rank <= 128) hipLaunchKernelGGL((lora_down_kernel<XT, 8, 4, MANY>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((lora_down_kernel<XT, 16, 2, MANY>), grid, dim3(128), 0, st, p);
}

template <bool VEC, bool MANY, bool FEW>
static void launch_up(const LoraArgs& p, hipStream_t st) {
    const dim3 grid((unsigned)((p.nrows + kUpRows - 1) / kUpRows), (unsigned)(p.ntok / kUpTokens + p.nseg));
    const size_t lds = (size_t)((p.max_rank + 15) / 16) * 96 * kUpTokens;  // three parts of every token's inner values
    if (p.split == 8) hipLaunchKernelGGL((lora_up_kernel<8, VEC, MANY, FEW>), grid, dim3(256), lds, st, p);
    else if (p.split == 2) hipLaunchKernelGGL((lora_up_kernel<2, VEC, MANY, FEW>), grid, dim3(256), lds, st, p);
    else hipLaunchKernelGGL((lora_up_kernel<1, VEC, MANY, FEW>), grid, dim3(256), lds, st, p);
}

extern "C" int qmm_lora(int xtype, const void* x, int64_t ldx, int64_t ntok, int64_t k, const uint16_t* a, const uint16_t* b,
                        const int32_t* ranks, const float* scales, int nadapters, int max_rank, const int32_t* seg_off,
                        const int32_t* seg_adapter, int nseg, const float* base, int64_t ldbase, float* y, int64_t ldy,
                        int64_t nrows, void* ws, size_t ws_bytes, void* stream) {
    if ((xtype != QMM_TYPE_F16 && xtype != QMM_TYPE_F32) || ntok < 0 || k < 32 || k % 32 || ldx < k || nadapters < 1 || max_rank < 8 ||
        max_rank % 8 || nseg < 0 || nrows < 1 || ldbase < nrows || ldy < nrows)
        return QMM_EINVAL;
    if (k > kMaxK || max_rank > kLoraMaxRank || ntok > kLoraMaxTokens || nseg > kLoraMaxSegments || nrows > 0x7FFFFF00 || ldbase > 0x7FFFFFFF || ldy > 0x7FFFFFFF)
        return QMM_EUNSUPPORTED;
    if (ntok == 0 || nseg == 0) return QMM_OK;
    if (!x || !a || !b || !ranks || !scales || !seg_off || !seg_adapter || !base || !y || !ws) return QMM_EINVAL;
    if (base == y && ldbase != ldy) return QMM_EINVAL;
    if (!aligned(x, 16) || ldx * (int64_t)type_bytes(xtype) % 16 || !aligned(a, 16) || !aligned(b, 16) || !aligned(ranks, 4) ||
        !aligned(scales, 4) || !aligned(seg_off, 4) || !aligned(seg_adapter, 4) || !aligned(base, 4) || !aligned(y, 4) || !aligned(ws, 16))
        return QMM_EALIGN;
    if (ws_bytes < qmm_lora_workspace(ntok, max_rank)) return QMM_ESPACE;
    LoraArgs p{x, a, b, ranks, seg_off, seg_adapter, scales, base, y, (float*)ws, ldx, ldbase, ldy, (int)ntok, (int)k,
               nadapters, max_rank, nseg, (int)nrows, lora_split(ntok)};
    const hipStream_t st = as_stream(stream);
    const bool many = nseg > 64;
    if (xtype == QMM_TYPE_F32) many ? launch_down<kF32, true>(p, st) : launch_down<kF32, false>(p, st);
    else many ? launch_down<kBin16, true>(p, st) : launch_down<kBin16, false>(p, st);
    // y and base 8 bytes at a time
    const bool vec = aligned(base, 8) && aligned(y, 8) && ldbase % 2 == 0 && ldy % 2 == 0 && nrows % 2 == 0;
    const bool few = ntok <= 8 * (int64_t)nseg;  // tiles of up to 8 tokens on average
    if (vec && many) few ? launch_up<true, true, true>(p, st) : launch_up<true, true, false>(p, st);
    else if (vec) few ? launch_up<true, false, true>(p, st) : launch_up<true, false, false>(p, st);
    else if (many) few ? launch_up<false, true, true>(p, st) : launch_up<false, true, false>(p, st);
    else few ? launch_up<false, false, true>(p, st) : launch_up<false, false, false>(p, st);
    return launch_status();
}
