// cache8.cu -- the paged 8-bit K/V cache: rows in (quantised), rows out, and
// copies of pages.  All three are HBM-bound and make one pass over their data.
//
// Quantisation.  The scale of a (block of tokens, head) is the smallest power
// of two s with max |x| <= s X over the finite values x of its rows, X = 448
// (e4m3) or 127 (int8), never below 2^-126, and 0 when all are 0; a value
// becomes the 8-bit value nearest x / s, ties to even.  With a power of two
// the division is exact, so the stored value has one rounding, and e4m3, which
// has an exponent of its own, loses nothing against an arbitrary scale but one
// binade at the small end.
#include <cmath>

#include "cache8.cuh"

namespace gqa {

int check_cache8(const Cache8 &c, bool need_ptrs) {
    if (c.kind != GQA_E4M3 && c.kind != GQA_INT8)
        return set_error(GQA_ERR_INVALID_ARG, "kind=%d must be GQA_E4M3 or GQA_INT8", c.kind);
    if (c.Hkv < 1) return set_error(GQA_ERR_INVALID_ARG, "Hkv=%d must be >= 1", c.Hkv);
    if (c.d < 1) return set_error(GQA_ERR_INVALID_ARG, "head dim d=%d must be >= 1", c.d);
    if (c.d != 64 && c.d != 128)
        return set_error(GQA_ERR_UNSUPPORTED, "head dim d=%d: the 8-bit cache supports 64 and 128", c.d);
    if (c.n_pages < 1) return set_error(GQA_ERR_INVALID_ARG, "n_pages=%d must be >= 1", c.n_pages);
    if (c.page < kC8Rows || c.page % kC8Rows || c.page > kC8MaxPage)
        return set_error(GQA_ERR_INVALID_ARG, "page=%d must be a multiple of %d in [%d, %d]", c.page,
                         kC8Rows, kC8Rows, kC8MaxPage);
    if (c.block < kC8Rows || c.block % kC8Rows || c.block > kC8MaxBlock || c.page % c.block)
        return set_error(GQA_ERR_INVALID_ARG,
                         "block=%d must be a multiple of %d, at most %d, that divides page=%d",
                         c.block, kC8Rows, kC8MaxBlock, c.page);
    // rows of the cache are numbered by ints
    if (static_cast<double>(c.n_pages) * c.Hkv * c.page > 2147483647.0)
        return set_error(GQA_ERR_UNSUPPORTED, "n_pages=%d x Hkv=%d x page=%d exceeds 2^31 - 1 rows",
                         c.n_pages, c.Hkv, c.page);
    if (!need_ptrs) return GQA_OK;
    if (int rc = check_ptr(c.k, 16, "k_cache")) return rc;
    if (int rc = check_ptr(c.v, 16, "v_cache")) return rc;
    if (int rc = check_ptr(c.k_scale, 4, "k_scale")) return rc;
    return check_ptr(c.v_scale, 4, "v_scale");
}

int check_table(int B, int M, int page) {
    if (B < 0 || M < 1)
        return set_error(GQA_ERR_INVALID_ARG, "B=%d must be >= 0 and M=%d page slots >= 1", B, M);
    if (static_cast<long long>(M) * page > 0x7fffffffLL - kC8MaxPage)
        return set_error(GQA_ERR_UNSUPPORTED, "M=%d x page=%d rows exceed an int", M, page);
    return GQA_OK;
}

// ------------------------------------------------------------------ append --
//
// Unit: the rows that one call adds to one (sequence, block, K/V head) of K or
// V, handled by min(block, T) * d / 64 threads, in whole warps, that hold the unit's
// new values in registers (up to 8 16-byte loads each, all in flight; 4 for at most 16
// rows of 64): largest magnitude, scale, quantise, store.  Rows of the block from
// earlier calls are read only when the scale grows.  Units of neighbouring heads share
// a CTA of 256 threads, so a CTA reads whole runs of the [B, T, Hkv, d] input.  At most
// 64 registers a thread keep four such CTAs on an SM.
//
// Measured on a B200, 8 prompts of 1024-4096 rows, 8 heads, d = 128 (126 MB): int8,
// blocks of 64: 22 us, 88 % of the copy rate; e4m3, blocks of 16: 21 us, 94 %.  One row
// of each of 64 sequences: 3.0 us, a launch and four dependent loads.  Steps on the
// first: 48 us; loads before the page lookup and a barrier per unit 37; int8 rounding
// by one addition 35; CTAs of 256 threads 28 (512: 39), 64 registers 25; the
// conversion of infinities and NaN out of the way 23; grid indices in place of
// divisions 22.

struct ApParams {
    Cache8 c;
    const uint4 *k_new, *v_new;
    const int32_t *table, *seqlens, *counts;
    int T, M, nblk;                      // nblk: scale blocks of a page
    int *status;
};

template <bool kInt8>
__device__ __forceinline__ float scale_for(uint32_t amax_bits) {
    if (amax_bits == 0) return 0.0f;
    // amax = 1.m 2^e:  448 = 1.75 2^8, 127 = 1.984375 2^6
    const int e = static_cast<int>(amax_bits >> 23) - 127;
    const uint32_t m = amax_bits & 0x7fffffu;
    const int x = kInt8 ? e - 6 + (m > 0x7e0000u) : e - 8 + (m > 0x600000u);
    return __uint_as_float(static_cast<uint32_t>(max(x, -126) + 127) << 23);
}

template <int D, bool kInt8, int kPasses>
__global__ void __launch_bounds__(512, 2)
cache8_append_kernel(const ApParams p) {
    dependents_may_launch();
    wait_for_stream();
    constexpr int kC = D / 8;                       // 16-byte columns of an input row
    __shared__ uint32_t s_max[2][16];               // one per warp; [1]: finite values only
    // CTA: the units threadIdx.y of (K or V, head) number blockIdx.x * blockDim.y + ..., of
    // the blockIdx.y-th block that the call can touch, of sequence blockIdx.z
    const int slot = threadIdx.y, tid = threadIdx.x, n_unit = blockDim.x, b = blockIdx.z;
    const int uh = blockIdx.x * blockDim.y + slot, kv = uh >= p.c.Hkv, h = uh - (kv ? p.c.Hkv : 0);
    if (uh >= 2 * p.c.Hkv) return;                  // whole units: they share no barrier
    const int block = p.c.block, start = p.seqlens[b];
    int count = p.counts ? p.counts[b] : p.T;
    const bool bad = start < 0 || start > p.M * p.c.page || count < 0 || count > p.T;
    const int skip = start % block;                 // older rows of the first block
    const int t0 = static_cast<int>(blockIdx.y) * block - skip;  // new row of the block's first row
    if (!bad && (t0 >= count || count == 0)) return;             // no new row (count 0 in mid-block)
    if (bad) count = t0;                            // no rows
    const int r0 = max(0, -t0), r1 = min(block, count - t0);

    // new rows r0 .. r1 - 1 -> registers; thread tid holds column tid % kC of every step-th
    const int col = tid % kC, row = tid / kC, step = n_unit / kC;
    const uint4 *src = (kv ? p.v_new : p.k_new) +
                       ((static_cast<size_t>(b) * p.T + t0 + r0 + row) * p.c.Hkv + h) * kC + col;
    const size_t stride = static_cast<size_t>(step) * p.c.Hkv * kC;
    uint4 x[kPasses];
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r0 + row + j * step < r1) x[j] = src[j * stride];
    }
    int page = -1, r_page = 0;
    if (!bad) {
        const uint32_t pos0 = static_cast<uint32_t>(start) + t0, s = pos0 / p.c.page;
        r_page = pos0 - s * p.c.page;
        if (s < static_cast<uint32_t>(p.M)) page = p.table[static_cast<size_t>(b) * p.M + s];
    }
    if (page < 0 || page >= p.c.n_pages) {          // the whole unit
        if (tid == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
        return;
    }
    const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
    float *scale = (kv ? p.c.v_scale : p.c.k_scale) + ph * p.nblk + r_page / block;
    const float s_old = r0 > 0 ? *scale : 0.0f;

    auto hmax = [](uint32_t a, uint32_t w) {        // NaN if either is
        const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
        return *reinterpret_cast<const uint32_t *>(&r);
    };
    const int unit_warps = n_unit / 32;
    auto unit_sync = [&]() {
        if (unit_warps > 1) named_barrier_sync(1 + slot, n_unit);
        else __syncwarp();
    };
    // largest fp32 magnitude of the unit, as bits, from each thread's two bf16 magnitudes
    auto unit_max = [&](uint32_t v, uint32_t (&s)[16]) {
        uint32_t m = __reduce_max_sync(0xffffffffu, max(v << 16, v & 0xffff0000u));
        if (unit_warps > 1) {
            if ((tid & 31) == 0) s[slot * unit_warps + (tid >> 5)] = m;
            unit_sync();
            for (int w = 0; w < unit_warps; ++w) m = max(m, s[slot * unit_warps + w]);
        }
        return m;
    };
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < kPasses; ++j)
        mx = hmax(hmax(hmax(hmax(mx, x[j].x), x[j].y), x[j].z), x[j].w);
    uint32_t amax = unit_max(mx, s_max[0]);
    const bool special = amax >= 0x7f800000u;       // infinities or NaN among the new values
    if (special) {
        // the largest finite value counts; with infinities, at least the smallest one
        uint32_t fin = 0;
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
                if (lo <= 0x7f80u) fin = max(fin, lo < 0x7f80u ? lo : 1u);
                if (hi <= 0x7f80u) fin = max(fin, hi < 0x7f80u ? hi : 1u);
            }
        }
        amax = unit_max(fin, s_max[1]);
    }
    const float s = fmaxf(scale_for<kInt8>(amax), s_old);
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    uint2 *dst = reinterpret_cast<uint2 *>(kv ? p.c.v : p.c.k) + (ph * p.c.page + r_page) * kC + col;
    auto store = [&](auto convert) {
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            const int r = r0 + row + j * step;
            const float2 a = bf16x2_to_float2(x[j].x), c = bf16x2_to_float2(x[j].y);
            const float2 e = bf16x2_to_float2(x[j].z), g = bf16x2_to_float2(x[j].w);
            const uint2 w = make_uint2(convert(a.x * inv, a.y * inv, c.x * inv, c.y * inv),
                                       convert(e.x * inv, e.y * inv, g.x * inv, g.y * inv));
            if (r < r1) dst[r * kC] = w;
        }
    };
    if (special)
        store([](float a, float b, float c, float d) { return from_f32x4<kInt8>(a, b, c, d); });
    else
        store([](float a, float b, float c, float d) { return from_small_f32x4<kInt8>(a, b, c, d); });
    if (s > s_old)                                  // older rows: to the larger scale
        for (int r = row; r < r0; r += step) {
            const uint2 w = dst[r * kC];
            float f[4], g[4];
            to_f32x4<kInt8>(w.x, f);
            to_f32x4<kInt8>(w.y, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = f[e] * s_old * inv;
                g[e] = g[e] * s_old * inv;
            }
            dst[r * kC] = make_uint2(from_small_f32x4<kInt8>(f[0], f[1], f[2], f[3]),
                                     from_small_f32x4<kInt8>(g[0], g[1], g[2], g[3]));
        }
    if (r0 > 0) unit_sync();                        // every thread has read s_old
    if (tid == 0) *scale = s;
}

// -------------------------------------------------------------------- read --
//
// One warp per (16 rows, K/V head) of K or V: the rows lie in one page and one
// scale block, 16 d contiguous bytes.  All loads are in flight before the first
// conversion; a value byte * scale has at most 8 significant bits and is exact
// in bf16 for power-of-two scales.  Measured on a B200: 8 sequences of 4096-8192 rows,
// 8 heads, d = 128: 60 us, 95 % of the copy rate; one of 1000 rows 3.4 us.

struct RdParams {
    Cache8 c;
    const int32_t *table, *seqlens;
    uint4 *k_out, *v_out;
    int B, T, M, n_grp;                 // n_grp: groups of 16 rows in T
    long long n_warps;
    int *status;
};

template <int D, bool kInt8>
__global__ void __launch_bounds__(256)
cache8_read_kernel(const RdParams p) {
    dependents_may_launch();
    wait_for_stream();
    constexpr int kC = D / 8, kRows = 32 / kC, kN = kC8Rows / kRows;   // 8 bytes in, 16 out per lane
    const long long u = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (u >= p.n_warps) return;
    const int lane = threadIdx.x & 31;
    long long x = u;
    const int h = static_cast<int>(x % p.c.Hkv);
    x /= p.c.Hkv;
    const int kv = static_cast<int>(x & 1);
    x >>= 1;
    const int t0 = static_cast<int>(x % p.n_grp) * kC8Rows;
    const int b = static_cast<int>(x / p.n_grp);
    int L = p.seqlens[b];
    if (L < 0 || L > p.M * p.c.page) {
        if (lane == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
        L = L < 0 ? 0 : p.M * p.c.page;
    }
    int page = -1;
    if (t0 < L) {
        page = p.table[static_cast<size_t>(b) * p.M + t0 / p.c.page];
        if (page < 0 || page >= p.c.n_pages) {
            if (lane == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
            page = -1;
        }
    }
    const int row = lane / kC, col = lane % kC;
    uint2 w[kN];
    float s = 0.0f;
    if (page >= 0) {
        const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
        const int r = t0 % p.c.page;
        s = (kv ? p.c.v_scale : p.c.k_scale)[ph * (p.c.page / p.c.block) + r / p.c.block];
        const uint2 *src = reinterpret_cast<const uint2 *>(kv ? p.c.v : p.c.k) + (ph * p.c.page + r) * kC;
#pragma unroll
        for (int j = 0; j < kN; ++j) w[j] = src[j * 32 + lane];
    }
    uint4 *dst = (kv ? p.v_out : p.k_out) + ((static_cast<size_t>(b) * p.T + t0) * p.c.Hkv + h) * kC + col;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int t = j * kRows + row;
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0 && t0 + t < L) {
            float f[4], g[4];
            to_f32x4<kInt8>(w[j].x, f);
            to_f32x4<kInt8>(w[j].y, g);
            o = make_uint4(pack_bf16x2(f[0] * s, f[1] * s), pack_bf16x2(f[2] * s, f[3] * s),
                           pack_bf16x2(g[0] * s, g[1] * s), pack_bf16x2(g[2] * s, g[3] * s));
        }
        if (t0 + t < p.T) dst[static_cast<size_t>(t) * p.c.Hkv * kC] = o;
    }
}

// -------------------------------------------------------------------- copy --
//
// moves [1 + cap, 3]: row 0 holds the number of moves, the others (source page,
// destination page, rows).  One CTA per (move, K or V, head), grid-stride: the
// rows of a head in a page are contiguous.  Measured on a B200: 1277 pages of 128 KB
// 55 us, 94 % of the copy rate; 79 half pages 3.3 us.

struct CpParams {
    Cache8 c;
    const int32_t *moves;
    int cap;
    int *status;
};

constexpr int kCpThreads = 128, kCpBatch = 4;

__global__ void __launch_bounds__(kCpThreads)
cache8_copy_kernel(const CpParams p) {
    dependents_may_launch();
    wait_for_stream();
    int n = p.moves[0];
    if (n < 0 || n > p.cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
        n = n < 0 ? 0 : p.cap;
    }
    const long long units = 2ll * n * p.c.Hkv;
    const int nblk = p.c.page / p.c.block;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int h = static_cast<int>(u % p.c.Hkv);
        const int kv = static_cast<int>(u / p.c.Hkv) & 1;
        const int32_t *mv = p.moves + 3 * (1 + u / p.c.Hkv / 2);
        const int a = mv[0], b = mv[1], rows = mv[2];
        if (a < 0 || a >= p.c.n_pages || b < 0 || b >= p.c.n_pages || rows < 0 || rows > p.c.page) {
            if (threadIdx.x == 0) record_status(p.status, GQA_ERR_INVALID_ARG);
            continue;
        }
        const size_t from = static_cast<size_t>(a) * p.c.Hkv + h, to = static_cast<size_t>(b) * p.c.Hkv + h;
        const int row16 = p.c.d / 16;
        uint4 *base = static_cast<uint4 *>(kv ? p.c.v : p.c.k);
        const uint4 *src = base + from * p.c.page * row16;
        uint4 *dst = base + to * p.c.page * row16;
        const int words = rows * row16;
        float *scale = kv ? p.c.v_scale : p.c.k_scale;
        float s = 0.0f;
        const bool has_s = threadIdx.x < (rows + p.c.block - 1) / p.c.block;
        if (has_s) s = scale[from * nblk + threadIdx.x];
        for (int i = threadIdx.x; i < words; i += kCpThreads * kCpBatch) {
            uint4 v[kCpBatch];
#pragma unroll
            for (int x = 0; x < kCpBatch; ++x)
                if (i + x * kCpThreads < words) v[x] = src[i + x * kCpThreads];
#pragma unroll
            for (int x = 0; x < kCpBatch; ++x)
                if (i + x * kCpThreads < words) dst[i + x * kCpThreads] = v[x];
        }
        if (has_s) scale[to * nblk + threadIdx.x] = s;
    }
}
static_assert(kC8MaxPage / kC8Rows <= kCpThreads, "one thread per scale of a page");

}  // namespace gqa

using namespace gqa;

extern "C" int gqa_cache8_append(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                                 const int32_t *table, const int32_t *seqlens,
                                 const int32_t *counts, const void *k, const void *v, int kind, int B,
                                 int T, int M, int n_pages, int Hkv, int page, int d, int block,
                                 gqa_stream_t stream) {
    clear_error();
    ApParams p;
    p.c = {k_cache, v_cache, k_scale, v_scale, kind, n_pages, Hkv, page, d, block};
    if (int rc = check_cache8(p.c, B > 0 && T > 0)) return rc;
    if (int rc = check_table(B, M, page)) return rc;
    if (T < 0 || T > 0x7fffffff - 2 * kC8MaxBlock)
        return set_error(GQA_ERR_INVALID_ARG, "T=%d must be >= 0 and leave room for a block", T);
    if (B == 0 || T == 0) return GQA_OK;
    const int n_blk = (T + block - 2) / block + 1;  // blocks that T rows can touch
    if (n_blk > 65535 || B > 65535)
        return set_error(GQA_ERR_UNSUPPORTED, "cache8_append: T=%d rows in %d blocks or B=%d exceed 65535", T,
                         n_blk, B);
    if (int rc = check_ptr(k, 16, "k")) return rc;
    if (int rc = check_ptr(v, 16, "v")) return rc;
    if (int rc = check_ptr(table, 4, "table")) return rc;
    if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
    if (counts)
        if (int rc = check_ptr(counts, 4, "counts")) return rc;
    if (int rc = require_sm100()) return rc;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    p.k_new = static_cast<const uint4 *>(k);
    p.v_new = static_cast<const uint4 *>(v);
    p.table = table;
    p.seqlens = seqlens;
    p.counts = counts;
    p.T = T;
    p.M = M;
    p.nblk = page / block;
    const int most = T < block ? T : block;         // new rows of a unit at most
    const int unit = (most * d / 64 + 31) / 32 * 32;             // whole warps
    const int per_cta = unit >= 256 ? 1 : 256 / unit;
    const int n_x = (2 * Hkv - 1) / per_cta + 1;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool int8 = kind == GQA_INT8;
    auto kern = d == 128     ? (int8 ? cache8_append_kernel<128, true, 8> : cache8_append_kernel<128, false, 8>)
                : most <= 16 ? (int8 ? cache8_append_kernel<64, true, 4> : cache8_append_kernel<64, false, 4>)
                             : (int8 ? cache8_append_kernel<64, true, 8> : cache8_append_kernel<64, false, 8>);
    return launch_dependent(kern, dim3(n_x, n_blk, B), dim3(unit, per_cta), 0, s,
                            "cache8_append_kernel launch", p);
}

extern "C" int gqa_cache8_read(const void *k_cache, const void *v_cache, const float *k_scale,
                               const float *v_scale, const int32_t *table, const int32_t *seqlens,
                               void *k, void *v, int kind, int B, int T, int M, int n_pages, int Hkv,
                               int page, int d, int block, gqa_stream_t stream) {
    clear_error();
    RdParams p;
    p.c = {const_cast<void *>(k_cache), const_cast<void *>(v_cache), const_cast<float *>(k_scale),
           const_cast<float *>(v_scale), kind, n_pages, Hkv, page, d, block};
    if (int rc = check_cache8(p.c, B > 0 && T > 0)) return rc;
    if (int rc = check_table(B, M, page)) return rc;
    if (T < 0 || T > 0x7fffffff - kC8Rows)
        return set_error(GQA_ERR_INVALID_ARG, "T=%d must be >= 0 and leave room for 16 rows", T);
    if (B == 0 || T == 0) return GQA_OK;
    if (int rc = check_ptr(k, 16, "k")) return rc;
    if (int rc = check_ptr(v, 16, "v")) return rc;
    if (int rc = check_ptr(table, 4, "table")) return rc;
    if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
    if (int rc = require_sm100()) return rc;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    p.table = table;
    p.seqlens = seqlens;
    p.k_out = static_cast<uint4 *>(k);
    p.v_out = static_cast<uint4 *>(v);
    p.B = B;
    p.T = T;
    p.M = M;
    p.n_grp = (T + kC8Rows - 1) / kC8Rows;
    p.n_warps = 2ll * Hkv * p.n_grp * B;
    const long long ctas = (p.n_warps + 7) / 8;
    if (ctas > 0x7fffffffLL) return set_error(GQA_ERR_UNSUPPORTED, "cache8_read grid too large");
    const unsigned grid = static_cast<unsigned>(ctas);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool int8 = kind == GQA_INT8;
    auto kern = d == 128 ? (int8 ? cache8_read_kernel<128, true> : cache8_read_kernel<128, false>)
                         : (int8 ? cache8_read_kernel<64, true> : cache8_read_kernel<64, false>);
    return launch_dependent(kern, grid, 256, 0, s, "cache8_read_kernel launch", p);
}

extern "C" int gqa_cache8_copy(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                               const int32_t *moves, int cap, int n_pages, int Hkv, int page, int d,
                               int block, gqa_stream_t stream) {
    clear_error();
    CpParams p;
    p.c = {k_cache, v_cache, k_scale, v_scale, GQA_INT8, n_pages, Hkv, page, d, block};
    if (cap < 0) return set_error(GQA_ERR_INVALID_ARG, "cap=%d moves must be >= 0", cap);
    if (int rc = check_cache8(p.c, cap > 0)) return rc;
    if (cap == 0) return GQA_OK;
    if (int rc = check_ptr(moves, 4, "moves")) return rc;
    if (int rc = require_sm100()) return rc;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    p.moves = moves;
    p.cap = cap;
    int n_sm = 0;
    if (int rc = sm_count(&n_sm)) return rc;
    const long long units = 2ll * cap * Hkv, full = 16ll * n_sm;
    return launch_dependent(cache8_copy_kernel, static_cast<unsigned>(units < full ? units : full), kCpThreads,
                            0, reinterpret_cast<cudaStream_t>(stream), "cache8_copy_kernel launch", p);
}
