// decode8.cu -- split-KV grouped-query decode over a paged 8-bit K/V cache.
//
//   s_j = scale <q, k_j>,  o = sum_j softmax(s)_j v_j,  k_j, v_j = byte * scale of its block
//
// HBM-bound: the cache is read once, 2 d bytes per key and K/V head, and the
// grid has to keep that stream going.  One CTA per (split, K/V head, sequence);
// its four warps take 32-key tiles in turn, each with a TMA ring of its own: one
// lane issues a box per page piece (32 or 16 keys, whatever divides the page),
// 128-byte swizzle, and no warp waits for another before the end of the split.
// A lane holds the page and the scales of one 16-key group of its warp's tiles.
//
// Arithmetic per byte is what competes with the stream, so the products are laid
// out for few instructions:
//   - S^T = K Q^T and O^T = V^T P^T as m16n8k16 f16 products with the keys (or
//     the elements of V) as the M rows and the G = Hq / Hkv query heads of the
//     group as the N columns, 8 at a time: with the heads as M rows, three
//     quarters of each product, softmax and rescaling would be padding for G = 4.
//   - e4m3 and int8 values are exact in f16, so K and V need no scaling to enter
//     a product; q (8 significant bits) is multiplied by a power of two per row
//     to sit at 1 and is exact in f16 down to 2^-14 of the row's largest value,
//     and absolutely to 2^-25 of it below.  The 16 keys of a group lie in one
//     scale block: the K scale multiplies the scores, the V scale the weights.
//   - both operands come straight from shared memory as 16-byte loads: the
//     contraction index of Q K^T may be permuted, so a thread's K fragments are
//     the 32 consecutive bytes (d = 128) it loads; V's four keys per thread are
//     paired by byte permutes before the conversion.  P^T is S^T transposed by
//     movmatrix, 8 x 8 f16 at a time.
// The running maximum, sums and O stay in fp32; the weights enter the second
// product in f16 (11 significant bits, at most 2^-12 off).
//
// V scales.  O is kept in units of vref, a running reference of the V scales
// seen by the warp.  A block whose scale lies in [vref / 64, vref] multiplies
// its weights by scale / vref before they are rounded to f16 (they keep full
// precision down to 2^-8); any other scale becomes the new vref and O is
// rescaled, as for a new maximum.  vref never falls by more than 2^64 at once,
// which keeps O finite; weights of a smaller block are below 2^-64 vref.
//
// The last split of a (sequence, K/V head) to arrive merges them all; the
// arrival words and the merge's formula are those of decode.cu.
#include <cmath>

#include "cache8.cuh"

namespace gqa {

constexpr int kD8Keys = 32;                        // keys per tile
constexpr int kD8Warps = 4;                        // each takes every fourth tile
constexpr int kD8Threads = kD8Warps * 32;
constexpr int kD8Stages = 2;                       // TMA ring of each warp, in tiles
constexpr int kD8MaxTiles = 32;                    // tiles per split at most
constexpr int kD8MinTiles = 4;
constexpr int kD8Ctas = 444;                       // 148 SMs x 3 resident CTAs
static_assert(kD8MaxTiles / kD8Warps * 2 <= 32, "a lane per 16-key group of a warp");

struct D8Params {
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int32_t *table, *seqlens;
    __nv_bfloat16 *o;
    float *part_o, *part_lse;
    unsigned long long *arrivals, call_id;
    int B, Hq, Hkv, M, n_pages, page, nblk, block, box;   // box: keys per TMA box
    int n_splits, window, sinks;
    float scale_log2;
    double log_theta;
    int *status;
};

template <int D, int NT>
struct D8Layout {
    static constexpr int kTileBytes = kD8Keys * D;          // K or V of one tile
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kD8Stages * kStageBytes;   // of one warp
    // the end-of-split merge reuses the rings: per warp 8 NT rows of O, m and l.
    // Four floats of padding after every D / 8 and at the end of a row spread
    // the 16-byte stores of a quarter warp over all banks.
    static constexpr int kRows = 8 * NT;
    static constexpr int kRowFloats = D + 32 + 4;
    static constexpr int kMergeBytes = kD8Warps * kRows * (kRowFloats + 2) * 4;
    static constexpr int kBytes =
        kD8Warps * kRingBytes > kMergeBytes ? kD8Warps * kRingBytes : kMergeBytes;
    static constexpr int kSmemBytes = kBytes + 1024;        // + alignment slack
};

// Tiles a sequence of L keys reads, in order: those of the sinks
// below the window, then those from the window's first key on.
struct D8Tiles {
    int lo, sinks;              // key j is visible iff j < L and (j >= lo or j < sinks)
    int n_sink, first, n;       // sink tiles, first window tile, tiles in all
    __host__ __device__ D8Tiles(int L, int window, int n_sinks) {
        lo = window > 0 && L > window ? L - window : 0;
        sinks = window > 0 ? n_sinks : 0;
        const int below = sinks < lo ? sinks : lo;
        n_sink = (below + kD8Keys - 1) / kD8Keys;
        first = lo / kD8Keys > n_sink ? lo / kD8Keys : n_sink;
        const int last = L / kD8Keys + (L % kD8Keys > 0);
        n = n_sink + (last > first ? last - first : 0);
    }
    __device__ int tile(int i) const { return i < n_sink ? i : first + (i - n_sink); }
};

// Tiles per split of a sequence with n tiles.  About kD8Ctas CTAs should run
// when all B sequences are this long; a split has kD8MinTiles to kD8MaxTiles
// tiles, and at most max_splits splits exist.
__host__ __device__ inline int d8_split_tiles(int n, long long rows, int max_splits) {
    long long t = (n * rows + kD8Ctas - 1) / kD8Ctas;
    t = t < kD8MinTiles ? kD8MinTiles : (t > kD8MaxTiles ? kD8MaxTiles : t);
    const int need = (n + max_splits - 1) / max_splits;
    const int per = t > need ? static_cast<int>(t) : need;
    const int splits = (n + per - 1) / per;
    return splits > 0 ? (n + splits - 1) / splits : 1;   // even splits
}

// Byte offset of 16-byte chunk c (of D / 16) of key row `key` in a stage tile:
// rows of 128 bytes hold one key (D = 128) or two (D = 64).
template <int D>
__device__ __forceinline__ uint32_t d8_off(int key, int c) {
    if constexpr (D == 128) return key * 128 + ((c ^ (key & 7)) << 4);
    const int row = key >> 1;
    return row * 128 + (((((key & 1) << 2) | c) ^ (row & 7)) << 4);
}

// Key (of the warp's 16) that column n of score tile nb stands for.  The four
// keys of a thread's weights are then rows whose V chunks lie in different banks.
template <int D>
__device__ __forceinline__ int d8_key(int nb, int n) {
    return D == 128 ? nb * 8 + n : 4 * (n >> 1) + 2 * nb + (n & 1);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Transpose of an 8 x 8 matrix of f16 held one pair per lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// NT: tiles of 8 query heads.  kRope: the query is rotated as it is loaded.
template <int D, int NT, bool kInt8, bool kRope>
__global__ void __launch_bounds__(kD8Threads, NT == 1 ? 3 : (NT == 2 ? 2 : 1))
decode8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const D8Params p) {
    using Lay = D8Layout<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full_bar[kD8Warps][kD8Stages];
    __shared__ int abort_flag, merger;

    const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.Hq / p.Hkv;
    const int Lmax = p.M * p.page;
    const int len = p.seqlens[b];
    int L = len;
    if (L > Lmax || L < 0) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
        L = L < 0 ? 0 : Lmax;
    }
    const D8Tiles seq(L, p.window, p.sinks);
    const int per = d8_split_tiles(seq.n, static_cast<long long>(p.B) * p.Hkv, gridDim.x);
    const int n_splits = (seq.n + per - 1) / per;
    const size_t grow0 = static_cast<size_t>(b) * p.Hq + static_cast<size_t>(kvh) * G;
    if (split >= n_splits) {
        // with no visible key at all split 0 writes the group's rows as zeros
        if (split == 0)
            for (int idx = threadIdx.x; idx < G * D / 8; idx += kD8Threads)
                reinterpret_cast<uint4 *>(p.o + grow0 * D)[idx] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i0 = split * per + warp;                           // this warp's first tile
    const int n_iter = (min(per, seq.n - split * per) - warp + kD8Warps - 1) / kD8Warps;
    auto seen = [&](int key0, int n) {                           // any of n keys visible
        return key0 < L && (key0 + n > seq.lo || key0 < seq.sinks);
    };

    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0) {
        for (int s = 0; s < kD8Stages; ++s) mbar_init(&full_bar[warp][s], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // lane i: page of the 16 keys that are half i & 1 of this warp's tile i >> 1
    int g_page = -1;
    float g_ks = 0.0f, g_vs = -1.0f;                             // V scale -1: not there
    const int g_key = seq.tile(i0 + (lane >> 1) * kD8Warps) * kD8Keys + (lane & 1) * 16;
    if ((lane >> 1) < n_iter && seen(g_key, 16)) {               // g_key < L: the slot exists
        g_page = p.table[static_cast<size_t>(b) * p.M + g_key / p.page];
        if (g_page < 0 || g_page >= p.n_pages) {
            record_status(p.status, GQA_ERR_INVALID_ARG);
            g_page = -1;
        }
    }
    __syncthreads();

    uint8_t *ring = smem + warp * Lay::kRingBytes;
    // Copies of tile t into its ring slot, counted on the slot's barrier.
    auto issue = [&](int t) {
        const int p0 = __shfl_sync(0xffffffffu, g_page, 2 * t);
        const int p1 = __shfl_sync(0xffffffffu, g_page, 2 * t + 1);
        if (lane == 0) {
            uint64_t *bar = &full_bar[warp][t % kD8Stages];
            uint8_t *kt = ring + (t % kD8Stages) * Lay::kStageBytes;
            uint8_t *vt = kt + Lay::kTileBytes;
            const int key0 = seq.tile(i0 + t * kD8Warps) * kD8Keys;
            // 128-byte row of a key; fits an int (checked on the host)
            auto row = [&](int page, int key) {
                return ((page * p.Hkv + kvh) * p.page + key % p.page) / (128 / D);
            };
            if (p.box == kD8Keys) {                              // both halves in one page
                const int page = max(p0, p1);
                mbar_expect_tx(bar, page >= 0 ? Lay::kStageBytes : 0);
                if (page >= 0) {
                    tma_load_2d(kt, &tm_k, bar, 0, row(page, key0));
                    tma_load_2d(vt, &tm_v, bar, 0, row(page, key0));
                }
            } else {
                mbar_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * (Lay::kStageBytes / 2));
                if (p0 >= 0) {
                    tma_load_2d(kt, &tm_k, bar, 0, row(p0, key0));
                    tma_load_2d(vt, &tm_v, bar, 0, row(p0, key0));
                }
                if (p1 >= 0) {
                    tma_load_2d(kt + Lay::kTileBytes / 2, &tm_k, bar, 0, row(p1, key0 + 16));
                    tma_load_2d(vt + Lay::kTileBytes / 2, &tm_v, bar, 0, row(p1, key0 + 16));
                }
            }
        }
        __syncwarp();
    };
    int issued = 0;
    for (; issued < min(n_iter, kD8Stages); ++issued) issue(issued);
    if (g_page >= 0) {
        const size_t at = (static_cast<size_t>(g_page) * p.Hkv + kvh) * p.nblk + g_key % p.page / p.block;
        g_ks = p.k_scale[at];
        g_vs = p.v_scale[at];
    }

    const int gq = lane >> 2, tq = lane & 3;        // quad, lane in quad
    // Query fragments (column gq of head tile nt).  Contraction step s multiplies
    // elements 4 s .. 4 s + 3 of each thread's quarter of the row (D / 4 elements).
    constexpr int kQ = D / 4;
    const __nv_bfloat16 *qg = p.q + grow0 * D + tq * kQ;
    uint32_t qb[NT][D / 16][2];
    float qs[NT][2];                                // score scale of heads 2 tq, 2 tq + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + gq;
#pragma unroll
        for (int s = 0; s < D / 16; s += 2) {
            const uint4 w = r < G ? *reinterpret_cast<const uint4 *>(qg + r * D + 4 * s)
                                  : make_uint4(0u, 0u, 0u, 0u);
            qb[nt][s][0] = w.x;
            qb[nt][s][1] = w.y;
            qb[nt][s + 1][0] = w.z;
            qb[nt][s + 1][1] = w.w;
        }
    }
    if constexpr (kRope) {
        __shared__ float2 rope_cs[D / 2];
        const int m = max(len - 1, 0);
        for (int i = threadIdx.x; i < D / 2; i += kD8Threads) {
            float cs, sn;
            rope_cos_sin(m, rope_turns(i, D / 2, p.log_theta), cs, sn);
            rope_cs[i] = make_float2(cs, sn);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const float2 c0 = rope_cs[tq * (kQ / 2) + 2 * s], c1 = rope_cs[tq * (kQ / 2) + 2 * s + 1];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                qb[nt][s][0] = rope_rotate_pair(qb[nt][s][0], c0.x, c0.y);
                qb[nt][s][1] = rope_rotate_pair(qb[nt][s][1], c1.x, c1.y);
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // bring the row's largest value into [1, 2); an infinite or zero row stays as it is
        float mx = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const float2 a = bf16x2_to_float2(qb[nt][s][0]), c = bf16x2_to_float2(qb[nt][s][1]);
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(c.x), fabsf(c.y))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = static_cast<int>(__float_as_uint(mx) >> 23);          // biased exponent
        const bool fit = e > 0 && e < 255;
        const uint32_t ex = min(e, 253);            // 2^(ex - 127) and its inverse are normal
        const float up = fit ? __uint_as_float((254 - ex) << 23) : 1.0f;
        const float down = (fit ? __uint_as_float(ex << 23) : 1.0f) * p.scale_log2;
        qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * tq);
        qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * tq + 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 a = bf16x2_to_float2(qb[nt][s][h]);
                qb[nt][s][h] = pack_f16x2(a.x * up, a.y * up);
            }
    }
    // O^T: product j, accumulator e is element (D / 8) gq + 2 j + (e >> 1) of head 2 tq + (e & 1)
    float oacc[NT][D / 16][4];
    float m_run[NT][2], l_run[NT][2];
    float vref = 0.0f, vinv = 0.0f;                 // O is in units of vref (0: O is still 0)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[nt][j][e] = 0.0f;
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.0f;
    }

    for (int t = 0; t < n_iter; ++t) {
        const int st = t % kD8Stages;
        // warp-uniform outcome: the products below are warp-collective
        if (!__all_sync(0xffffffffu, mbar_wait(&full_bar[warp][st], (t / kD8Stages) & 1, &abort_flag,
                                               p.status)))
            break;
        const uint8_t *kt = ring + st * Lay::kStageBytes;
        const uint8_t *vt = kt + Lay::kTileBytes;
        const int key0 = seq.tile(i0 + t * kD8Warps) * kD8Keys;
        float ks[2], vs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            ks[x] = __shfl_sync(0xffffffffu, g_ks, 2 * t + x);
            vs[x] = __shfl_sync(0xffffffffu, g_vs, 2 * t + x);
        }
        const bool all = key0 + kD8Keys <= L && (key0 >= seq.lo || key0 + kD8Keys <= seq.sinks) &&
                         vs[0] != -1.0f && vs[1] != -1.0f;
        auto visible = [&](int x, int nb, int n) {
            const int key = key0 + x * 16 + d8_key<D>(nb, n);
            return vs[x] != -1.0f && key < L && (key >= seq.lo || key < seq.sinks);
        };
        // ---- S^T = K Q^T: half x, accumulator e is key (e >> 1, gq), head 2 tq + (e & 1) ----
        float sacc[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[nt][x][e] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    kt + d8_off<D>(x * 16 + d8_key<D>(0, gq), tq * (D / 64) + c));
                const uint4 v = *reinterpret_cast<const uint4 *>(
                    kt + d8_off<D>(x * 16 + d8_key<D>(1, gq), tq * (D / 64) + c));
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t a[4];
                    to_f16x2<kInt8>(uw[s], a[0], a[2]);
                    to_f16x2<kInt8>(vw[s], a[1], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816_f16(sacc[nt][x], a, qb[nt][c * 4 + s][0], qb[nt][c * 4 + s][1]);
                }
            }
        // ---- V scales: weight factor of each half, and O's change of units before it ----
        float pscale[2], ratio[2] = {1.0f, 1.0f};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (vs[x] == 0.0f || vs[x] == -1.0f) {
                pscale[x] = 0.0f;
                continue;
            }
            if (!(vs[x] <= vref && vs[x] * 64.0f >= vref)) {
                const float nv = fmaxf(vs[x], vref * 5.42101086e-20f);      // 2^-64
                if (vref > 0.0f) ratio[x] = vref / nv;
                vref = nv;
                vinv = 1.0f / nv;
            }
            pscale[x] = vs[x] * vinv;
        }
        // ---- softmax step ----
        uint32_t pb[NT][2][2];
        float alpha[NT][2];
        bool moved = ratio[0] != 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float s[2][4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[x][e] = sacc[nt][x][e] * (qs[nt][e & 1] * ks[x]);
                    if (!all && !visible(x, e >> 1, gq)) s[x][e] = -INFINITY;
                    mx[e & 1] = fmaxf(mx[e & 1], s[x][e]);
                }
            float m_use[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 4));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 8));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
                const float m_new = fmaxf(m_run[nt][h], mx[h]);
                m_use[h] = (m_new == -INFINITY) ? 0.0f : m_new;
                alpha[nt][h] = fast_exp2(m_run[nt][h] - m_use[h]);
                moved |= alpha[nt][h] != 1.0f;
                m_run[nt][h] = m_new;
                l_run[nt][h] *= alpha[nt][h];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][e] = fast_exp2(s[x][e] - m_use[e & 1]);
                l_run[nt][0] += s[x][0] + s[x][2];
                l_run[nt][1] += s[x][1] + s[x][3];
                pb[nt][x][0] = transpose_8x8(pack_f16x2(s[x][0] * pscale[x], s[x][1] * pscale[x]));
                pb[nt][x][1] = transpose_8x8(pack_f16x2(s[x][2] * pscale[x], s[x][3] * pscale[x]));
            }
        }
        // most tiles move neither a maximum nor the V reference
        auto rescale = [&](int nt, float f0, float f1) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                oacc[nt][j][0] *= f0;
                oacc[nt][j][1] *= f1;
                oacc[nt][j][2] *= f0;
                oacc[nt][j][3] *= f1;
            }
        };
        if (__any_sync(0xffffffffu, moved))
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) rescale(nt, alpha[nt][0] * ratio[0], alpha[nt][1] * ratio[0]);
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x == 1 && ratio[1] != 1.0f)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) rescale(nt, ratio[1], ratio[1]);
            constexpr int kW = D / 32;              // words of V per key and thread
            uint32_t vw[4][kW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = x * 16 + d8_key<D>(k >> 1, 2 * tq + (k & 1));
                if constexpr (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(vt + d8_off<D>(key, gq));
                    vw[k][0] = w.x;
                    vw[k][1] = w.y;
                    vw[k][2] = w.z;
                    vw[k][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(
                        vt + d8_off<D>(key, gq >> 1) + (gq & 1) * 8);
                    vw[k][0] = w.x;
                    vw[k][1] = w.y;
                }
            }
            if (!all) {
                // rows that are not visible hold anything, NaN included: 0 weight times 0
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!visible(x, k >> 1, 2 * tq + (k & 1)))
#pragma unroll
                        for (int w = 0; w < kW; ++w) vw[k][w] = 0u;
            }
#pragma unroll
            for (int w = 0; w < kW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {       // elements 4 w + 2 h, 4 w + 2 h + 1
                    const uint32_t sel = h ? 0x7362 : 0x5140;
                    uint32_t a[4];
                    to_f16x2<kInt8>(__byte_perm(vw[0][w], vw[1][w], sel), a[0], a[1]);
                    to_f16x2<kInt8>(__byte_perm(vw[2][w], vw[3][w], sel), a[2], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816_f16(oacc[nt][2 * w + h], a, pb[nt][x][0], pb[nt][x][1]);
                }
        }
        __syncwarp();                               // the slot is read: refill it
        if (issued < n_iter) issue(issued++);
    }
    // after a time-out, the copies in flight land before the block exits
    if (abort_flag)
        for (int u = max(0, issued - kD8Stages); u < issued; ++u)
            mbar_wait(&full_bar[warp][u % kD8Stages], (u / kD8Stages) & 1, &abort_flag, p.status, 1000000ull);

    // ---- merge the four warps' partial softmax states ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l_run[nt][h] += __shfl_xor_sync(0xffffffffu, l_run[nt][h], 4);
            l_run[nt][h] += __shfl_xor_sync(0xffffffffu, l_run[nt][h], 8);
            l_run[nt][h] += __shfl_xor_sync(0xffffffffu, l_run[nt][h], 16);
        }
    __syncthreads();                                // every tile consumed: reuse the rings
    constexpr int kRows = Lay::kRows, kStride = Lay::kRowFloats;
    float *s_o = reinterpret_cast<float *>(smem);             // [warp][row][kStride]
    float *s_m = s_o + kD8Warps * kRows * kStride;            // [warp][row]
    float *s_l = s_m + kD8Warps * kRows;                      // [warp][row]
    auto column = [](int c) { return c + 4 * (c / (D / 8)); };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = nt * 8 + 2 * tq + h;
            float *dst = s_o + (warp * kRows + r) * kStride + column((D / 8) * gq);
#pragma unroll
            for (int j = 0; j < D / 16; j += 2)
                *reinterpret_cast<float4 *>(dst + 2 * j) =
                    make_float4(oacc[nt][j][h] * vref, oacc[nt][j][h + 2] * vref,
                                oacc[nt][j + 1][h] * vref, oacc[nt][j + 1][h + 2] * vref);
            if (gq == 0) {
                s_m[warp * kRows + r] = m_run[nt][h];
                s_l[warp * kRows + r] = l_run[nt][h];
            }
        }
    __syncthreads();
    const size_t plane = static_cast<size_t>(p.B) * p.Hq;
    for (int idx = threadIdx.x; idx < G * D / 4; idx += kD8Threads) {
        const int r = idx / (D / 4), c = idx % (D / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kD8Warps; ++w) M = fmaxf(M, s_m[w * kRows + r]);
        float wsum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kD8Warps; ++w) {
            // 0 for a warp with no key (M is -inf when none has any)
            const float f = M == -INFINITY ? 0.0f : fast_exp2(s_m[w * kRows + r] - M);
            const float4 x = *reinterpret_cast<const float4 *>(s_o + (w * kRows + r) * kStride + column(c));
            wsum += f * s_l[w * kRows + r];
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (n_splits == 1) {
            *reinterpret_cast<uint2 *>(p.o + (grow0 + r) * D + c) =
                make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        } else {
            const size_t at = split * plane + grow0 + r;
            *reinterpret_cast<float4 *>(p.part_o + at * D + c) = acc;
            if (c == 0) p.part_lse[at] = wsum == 0.0f ? -INFINITY : M + __log2f(wsum);
        }
    }
    if (n_splits == 1) return;

    // ---- the last split of this (sequence, K/V head) merges all of them ----
    // Arrival word: see decode.cu (call id and arrivals of that call).
    __threadfence();                                 // my partial rows, device-wide
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned long long *word = p.arrivals + static_cast<size_t>(b) * p.Hkv + kvh;
        unsigned long long cur = *reinterpret_cast<volatile unsigned long long *>(word), was, next;
        do {
            was = cur;
            next = (was >> 16) == p.call_id ? was + 1 : ((p.call_id << 16) | 1ull);
            cur = atomicCAS(word, was, next);
        } while (cur != was);
        const bool last = static_cast<int>(next & 0xFFFFu) == n_splits;
        if (last) *reinterpret_cast<volatile unsigned long long *>(word) = p.call_id << 16;
        merger = last;
    }
    __syncthreads();
    if (!merger) return;
    __threadfence();                                 // every split's partial rows are visible
    // One warp per head row; D / 4 lanes hold a row's columns, and the other half
    // of the warp (D = 64) takes every second split.
    constexpr int kLanes = D / 4, kSub = 32 / kLanes, kBatch = 8;
    const int sub = lane / kLanes, c = lane % kLanes * 4;
    for (int r = warp; r < G; r += kD8Warps) {
        const float *lse = p.part_lse + grow0 + r;
        const float *po = p.part_o + (grow0 + r) * D + c;
        float M = -INFINITY;
        for (int i = lane; i < n_splits; i += 32) M = fmaxf(M, __ldcg(lse + i * plane));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        if (M == -INFINITY) M = 0.0f;                // every weight is 0 then
        float wsum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = sub; i < n_splits; i += kSub * kBatch) {
            float l[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const int sp = i + x * kSub;
                const bool in = sp < n_splits;
                l[x] = in ? __ldcg(lse + sp * plane) : -INFINITY;
                v[x] = in ? __ldcg(reinterpret_cast<const float4 *>(po + sp * plane * D))
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const float w = fast_exp2(l[x] - M);
                wsum += w;
                acc.x += w * v[x].x;
                acc.y += w * v[x].y;
                acc.z += w * v[x].z;
                acc.w += w * v[x].w;
            }
        }
        if constexpr (kSub == 2) {
            wsum += __shfl_xor_sync(0xffffffffu, wsum, 16);
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
        }
        const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
        if (sub == 0)
            *reinterpret_cast<uint2 *>(p.o + (grow0 + r) * D + c) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
}

static long long d8_tiles(long long keys) { return (keys + kD8Keys - 1) / kD8Keys; }

// Splits of the grid: enough for any sequence of up to `tiles` tiles (a shorter
// one may use as many, since its splits are shorter).
static long long d8_max_splits(int B, int Hkv, long long tiles) {
    const long long rows = static_cast<long long>(B) * Hkv;
    const long long longest = (tiles + kD8MaxTiles - 1) / kD8MaxTiles;
    long long spread = (kD8Ctas + rows - 1) / rows;
    const long long most = (tiles + kD8MinTiles - 1) / kD8MinTiles;
    if (spread > most) spread = most;
    return longest > spread ? longest : spread;
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: partial O [splits, B, Hq, d] fp32 | partial lse [splits, B, Hq]
// fp32 (log2 units) | arrival words [B, Hkv] u64.
struct D8Workspace {
    size_t splits, off_lse, off_arrivals, bytes;
    D8Workspace(int B, int Hq, int Hkv, int d, long long Lmax) {
        splits = static_cast<size_t>(d8_max_splits(B, Hkv, d8_tiles(Lmax)));
        const size_t rows = splits * B * Hq;
        off_lse = align256(rows * d * sizeof(float));
        off_arrivals = off_lse + align256(rows * sizeof(float));
        bytes = splits > 1 ? off_arrivals + align256(static_cast<size_t>(B) * Hkv * 8) : 0;
    }
};

template <int D, int NT, bool kInt8, bool kRope>
static int launch_decode8_kernel(const CUtensorMap &tk, const CUtensorMap &tv, const D8Params &p,
                                 cudaStream_t stream) {
    auto kern = decode8_kernel<D, NT, kInt8, kRope>;
    const int smem = D8Layout<D, NT>::kSmemBytes;
    static CtxSlot setup;   // one per instantiation: the opt-in is set once per context
    if (int rc = once_per_context(setup, [&](int) {
            return check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   smem), "cudaFuncSetAttribute(decode8)");
        }))
        return rc;
    kern<<<dim3(p.n_splits, p.Hkv, p.B), kD8Threads, smem, stream>>>(tk, tv, p);
    return check_cuda(cudaGetLastError(), "decode8_kernel launch");
}

template <int D, int NT>
static int launch_decode8_kind(bool int8, bool rope, const CUtensorMap &tk, const CUtensorMap &tv,
                               const D8Params &p, cudaStream_t s) {
    if (int8)
        return rope ? launch_decode8_kernel<D, NT, true, true>(tk, tv, p, s)
                    : launch_decode8_kernel<D, NT, true, false>(tk, tv, p, s);
    return rope ? launch_decode8_kernel<D, NT, false, true>(tk, tv, p, s)
                : launch_decode8_kernel<D, NT, false, false>(tk, tv, p, s);
}

}  // namespace gqa

using namespace gqa;

extern "C" size_t gqa_decode8_workspace_size(int B, int Hq, int Hkv, int d, int Lmax) {
    if (B < 1 || Lmax < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1) return 0;
    return D8Workspace(B, Hq, Hkv, d, Lmax).bytes;
}

extern "C" int gqa_decode8(const void *q, const void *k_cache, const void *v_cache,
                           const float *k_scale, const float *v_scale, const int32_t *table,
                           const int32_t *seqlens, void *o, int kind, int B, int Hq, int Hkv, int d,
                           int M, int n_pages, int page, int block, int window, int sinks,
                           float scale, float theta, void *workspace, size_t workspace_bytes,
                           gqa_stream_t stream) {
    clear_error();
    if (int rc = check_heads(Hq, Hkv, d)) return rc;
    if (int rc = check_scale(scale)) return rc;
    const Cache8 c{const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                   const_cast<float *>(k_scale), const_cast<float *>(v_scale), kind, n_pages, Hkv,
                   page, d, block};
    if (int rc = check_cache8(c, B > 0)) return rc;
    if (int rc = check_table(B, M, page)) return rc;
    if (Hq / Hkv > 32)
        return set_error(GQA_ERR_UNSUPPORTED, "decode group size Hq/Hkv=%d exceeds 32", Hq / Hkv);
    if (window < 0 || sinks < 0)
        return set_error(GQA_ERR_INVALID_ARG, "window=%d and sinks=%d must be >= 0", window, sinks);
    if (theta != 0.0f)
        if (int rc = check_theta(theta)) return rc;
    if (B > 65535 || Hkv > 65535)
        return set_error(GQA_ERR_UNSUPPORTED, "decode8: B and Hkv must be <= 65535");
    if (B == 0) return GQA_OK;
    if (int rc = check_ptr(q, 16, "q")) return rc;
    if (int rc = check_ptr(o, 16, "o")) return rc;
    if (int rc = check_ptr(table, 4, "table")) return rc;
    if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
    const D8Workspace ws(B, Hq, Hkv, d, static_cast<long long>(M) * page);
    if (ws.splits > 0xFFFF)
        return set_error(GQA_ERR_UNSUPPORTED, "decode8: %d x %d rows give more than 65535 splits", M,
                         page);
    if (int rc = check_workspace(workspace, workspace_bytes, ws.bytes)) return rc;
    if (int rc = require_sm100()) return rc;
    D8Params p;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.seqlens = seqlens;
    p.o = static_cast<__nv_bfloat16 *>(o);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    p.part_o = reinterpret_cast<float *>(base);
    p.part_lse = reinterpret_cast<float *>(base + ws.off_lse);
    p.arrivals = reinterpret_cast<unsigned long long *>(base + ws.off_arrivals);
    p.call_id = next_call_id();
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.M = M;
    p.n_pages = n_pages;
    p.page = page;
    p.block = block;
    p.nblk = page / block;
    p.box = page % kD8Keys == 0 ? kD8Keys : 16;
    // a windowed sequence reads the tiles of its sinks and of its window
    long long tiles = d8_tiles(static_cast<long long>(M) * page);
    if (window > 0 && d8_tiles(window) + 1 + d8_tiles(sinks) < tiles)
        tiles = d8_tiles(window) + 1 + d8_tiles(sinks);
    p.n_splits = static_cast<int>(d8_max_splits(B, Hkv, tiles));
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.log_theta = theta > 0.0f ? log(static_cast<double>(theta)) : 0.0;
    const uint64_t rows = static_cast<uint64_t>(n_pages) * Hkv * page * d / 128;
    CUtensorMap tk, tv;
    if (int rc = encode_tmap_rows128(&tk, k_cache, rows, p.box * d / 128)) return rc;
    if (int rc = encode_tmap_rows128(&tv, v_cache, rows, p.box * d / 128)) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool int8 = kind == GQA_INT8, rope = theta > 0.0f;
    const int G = Hq / Hkv;
    if (d == 128)
        return G <= 8    ? launch_decode8_kind<128, 1>(int8, rope, tk, tv, p, s)
               : G <= 16 ? launch_decode8_kind<128, 2>(int8, rope, tk, tv, p, s)
                         : launch_decode8_kind<128, 4>(int8, rope, tk, tv, p, s);
    return G <= 8    ? launch_decode8_kind<64, 1>(int8, rope, tk, tv, p, s)
           : G <= 16 ? launch_decode8_kind<64, 2>(int8, rope, tk, tv, p, s)
                     : launch_decode8_kind<64, 4>(int8, rope, tk, tv, p, s);
}
