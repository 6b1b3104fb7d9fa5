// decode8.cu -- grouped-query decode over a paged 8-bit K/V cache.
//
//   s_j = scale <q, k_j>,  o = sum_j softmax(s)_j v_j,  k_j, v_j = byte * scale of its block
//
// HBM-bound: the cache is read once, 2 d bytes per key and K/V head, and the
// grid has to keep that stream going.  Work is counted in tiles of 32 keys.  The
// tiles of all units (sequence, K/V head), one after another, are cut into equal
// runs, one per CTA, with all CTAs resident at once: ragged lengths, few rows and
// many rows are balanced alike, a unit is cut into as few pieces as that allows,
// and a CTA starts and merges about once.  In the line of tiles each unit begins
// with a few empty places, which stand for the time that beginning a unit takes.
// Each CTA sums the places of all sequences to find its run.
//
// The four warps of a CTA take the tiles of a piece in turn, each with a TMA ring
// of its own: one lane issues a box per page part (32 or 16 keys, whatever divides
// the page), 128-byte swizzle, and no warp waits for another before the end of the
// piece.  A lane holds the page and the scales of one 16-key group of its warp's
// present 16 tiles, and those of the next 16, loaded that far ahead.
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
// product in f16: 11 significant bits, at most 2^-11 off, from 2^-14 up, and at
// most 2^-25 off below.  They are held, in the sums too, as 2^7 times themselves:
// the reference of a score is passed by less than 2^8, so that they fill f16's
// range to 2^15, and a weight keeps its precision down to 2^-21 of the largest.
//
// V scales.  O is kept in units of vref, a running reference of the V scales
// seen by the warp.  A block whose scale lies in [vref / 64, vref] multiplies
// its weights by scale / vref before they are rounded to f16 (they keep full
// precision down to 2^-15 of the largest); any other scale becomes the new vref and O is
// rescaled, as for a new maximum.  A vref that falls multiplies O, so it falls no
// further than leaves the largest element of O at 2^110: however often the scales
// fall, and whatever follows (at most 2^24 a key), O stays finite.  A fall cut
// short only loses blocks some 2^80 below what O, of any head, already holds.
//
// Groups of 17-32 heads are shared by two CTAs (blockIdx.y), which read the same run at
// the same time, once from HBM and once from L2.  With all 32 heads in one CTA the
// accumulators allow two CTAs per SM, a tile takes a warp twice as long and the merge has
// twice the rows: four sequences of 8192 keys, one K/V head, 24.2 us against 19.6; one of
// 1000, 13.7 against 10.1; 64 of 4608, eight K/V heads, 177 against 184.
//
// A unit that lies in one CTA's run is written by it.  Otherwise its pieces go to
// the workspace, and the last one to arrive merges them with the log-sum-exp
// identity.
//
// Measured on a B200, 8 K/V heads, d = 128 (share of the 6.47 TB/s copy rate): 64
// sequences of 1024-8192 keys, groups of 4: 103 us (93 %; on other cards up to 112); 64 of
// 4608, groups of 16: 107 us (88 %), of 32: 184 us (51 %, bound by the products: two CTAs
// convert each tile); a 2048-key window, int8: 51 us (79 %); two sequences of
// 100000-131072, groups of 8: 79 us (85 %); one sequence of 1024 keys: 7.3 us (bound by
// latency: three dependent loads, one tile a warp, a merge).  d = 64: 64 of 4608, groups of 4,
// 56 us (83 %), 128 of 8192 172 us (97 %); 68 sequences of 512 keys, 32 heads (five units
// per CTA, bound by what beginning a unit takes) 42.6 us (52 %).  Steps on
// the way, on the first of these: heads as M rows 176 us; keys as M rows 126; equal runs
// in place of splits of 1024 keys, seldom-moved reference, loads ahead of the copies 109;
// no retries at arrival, packed fp32 106; empty places 103-104.  Arrival as one addition
// with release and acquire, where two fences stood around it: 7.2 us against 7.5 for the
// one sequence, 79 against 81 for the two, 34.0 against 35.6 for two of 32768.
#include <climits>
#include <cmath>
#include <type_traits>

#include "cache8.cuh"
#include "decode8_runs.cuh"

namespace gqa {

constexpr int kD8Warps = 4;                        // each takes every fourth tile of a piece
constexpr int kD8Threads = kD8Warps * 32;
constexpr int kD8Epoch = 16;                       // tiles whose pages a warp's lanes hold
constexpr int kD8MinTiles = kD8Warps;              // shortest run of a CTA
constexpr float kD8Merge = 0.25f;                  // merging a piece, in tiles of a run
constexpr int kD8CtasPerSm = 3;                    // what shared memory and registers allow
constexpr int kD8MaxCtas = 148 * kD8CtasPerSm;     // all resident
constexpr int kD8Heads = 16;                       // query heads of a CTA at most
constexpr float kD8Least = -3.0e38f;               // reference of a row that has seen no key
constexpr float kD8Rescale = 8.0f;                 // log2 units: how far a score may pass the reference
constexpr float kD8Pieces = 10.0f;                 // pieces weigh at most 2^-10: a unit has fewer than 2^10
constexpr float kD8Lift = 7.0f;                    // weights in units of 2^-7: below 2^15, f16 holds 2^16
constexpr float kD8Room = 0x1p110f;                // a smaller vref makes O no larger than this
constexpr float kD8HalfTop = 0x1p28f;              // > 16 keys x 2^15 x 448, what half a tile adds

struct D8Params {
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int32_t *table, *seqlens;
    __nv_bfloat16 *o;
    float *part_o, *part_lse;                      // two pieces of `share` rows per CTA
    unsigned long long *arrivals, call_id;
    int B, Hq, Hkv, M, n_pages, page, nblk, box;          // box: keys per TMA box
    int share;                                     // heads of a group per CTA (blockIdx.y)
    unsigned long long page_inv;                   // ceil(2^35 / (page / 16))
    uint32_t block_inv;                            // ceil(2^16 / (block / 16))
    int window, sinks;
    float scale_log2;
    double log_theta;
    int *status;
};

template <int D, int NT>
struct D8Layout {
    static constexpr int kTileBytes = kD8Keys * D;          // K or V of one tile
    static constexpr int kStageBytes = 2 * kTileBytes;
    // TMA ring of one warp: 16 KB, with three CTAs per SM
    static constexpr int kStages = 2 * (128 / D);
    static constexpr int kRingBytes = kStages * kStageBytes;
    static_assert(kStages <= kD8Epoch, "copies run at most one epoch ahead");
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

// D (16x8, fp32) += A (16x16) B (16x8), f16 operands.
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Shared-memory loads at a 32-bit address plus a constant.
template <int kOff>
__device__ __forceinline__ void lds(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr), "n"(kOff));
}
template <int kOff>
__device__ __forceinline__ void lds(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2+%3];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(addr), "n"(kOff));
}

// 2-D tiled tensor load of whole 128-byte rows into shared memory, completion counted
// on bar; 32-bit shared-memory addresses.  No L2 hint: marking the stream evict-first
// saves 1-3 % when no page is shared, and costs 30 % when the sequences share theirs
// (64 of 8192 keys, four to a prefix: 178 us against 137).
__device__ __forceinline__ void copy_rows(uint32_t dst, const void *tmap, uint32_t bar, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(tmap), "r"(bar), "r"(0), "r"(row)
        : "memory");
}

// A unit's arrival word in global memory.
struct D8Word {
    unsigned long long *at;
    __device__ unsigned long long read() const { return *reinterpret_cast<volatile unsigned long long *>(at); }
    __device__ void set(unsigned long long x) const { *reinterpret_cast<volatile unsigned long long *>(at) = x; }
    __device__ void cas(unsigned long long from, unsigned long long to) const { atomicCAS(at, from, to); }
    __device__ unsigned long long add(unsigned long long x) const {      // release and acquire, device scope
        unsigned long long was;
        asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(was) : "l"(at), "l"(x) : "memory");
        return was;
    }
};

// Transpose of an 8 x 8 matrix of f16 held one pair per lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Largest finite magnitude in a warp's accumulators.
template <int NT, int N>
__device__ __forceinline__ float largest(const float (&acc)[NT][N][4]) {
    float top = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (fabsf(acc[nt][j][e]) < INFINITY) top = fmaxf(top, fabsf(acc[nt][j][e]));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// NT: tiles of 8 query heads.  kRope: the query is rotated as it is loaded.
template <int D, int NT, bool kInt8, bool kRope>
__global__ void __launch_bounds__(kD8Threads, kD8CtasPerSm)
decode8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const D8Params p) {
    using Lay = D8Layout<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int kStages = Lay::kStages;
    __shared__ uint64_t full_bar[kD8Warps][kStages];
    __shared__ int abort_flag[kD8Warps], merger;
    __shared__ __align__(16) float s_vref[kD8Warps];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;        // quad, lane in quad
    const int G = min(p.share, p.Hq / p.Hkv - static_cast<int>(blockIdx.y) * p.share);   // heads here
    const int cta = blockIdx.y * gridDim.x + blockIdx.x;
    const int Lmax = p.M * p.page;
    if (lane == 0) {
        abort_flag[warp] = 0;
        for (int s = 0; s < kStages; ++s) mbar_init(&full_bar[warp][s], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    // RoPE: the turns of each coordinate pair, while the stream's last kernel finishes
    __shared__ double rope_turn[kRope ? D / 2 : 1];
    if constexpr (kRope) {
        for (int i = threadIdx.x; i < D / 2; i += kD8Threads)
            rope_turn[i] = rope_turns(i, D / 2, p.log_theta);        // read by the same thread
    }
    dependents_may_launch();
    wait_for_stream();
    // places that each unit of sequence b takes in the line of tiles: kD8Begin empty
    // ones, then its tiles
    auto places_of = [&](int b) {
        const int n = D8Tiles(min(max(p.seqlens[b], 0), Lmax), p.window, p.sinks).n;
        return n > 0 ? n + kD8Begin : 0;
    };

    auto word_of = [&](size_t unit) { return D8Word{p.arrivals + unit * gridDim.y + blockIdx.y}; };

    // ---- this CTA's run of tiles; every warp finds it for itself ----
    int total = 0, longest = 0;                     // total fits an int (checked on the host)
    for (int b = lane; b < p.B; b += 32) {
        const int n = places_of(b);
        total += n;
        longest = max(longest, n);
    }
    total = __reduce_add_sync(0xffffffffu, total) * p.Hkv;
    // A unit of n tiles in runs of r has n / r pieces to merge, one after the other, for
    // r tiles read side by side by four warps: runs are not shorter than about
    // sqrt(n kD8Merge), in whole rounds of the warps.  (One unit of 32 heads, d = 64,
    // 60000 keys: 61 us with runs of 4 tiles at least, 31 so, 22 with the heads shared by two
    // CTAs since; 1024 keys in 8 units, 7.3.)
    const int least = static_cast<int>(sqrtf(kD8Merge * __reduce_max_sync(0xffffffffu, longest)));
    const int per = max((least + kD8Warps) / kD8Warps * kD8Warps,
                        (total - 1) / static_cast<int>(gridDim.x) + 1);
    D8Run run = {per * static_cast<int>(blockIdx.x), 0, 0, 0, 0};
    run.end = min(run.pos + per, total);
    // the unit it begins in
    if (run.pos < run.end)
        for (int b0 = 0, off = 0; b0 < p.B; b0 += 32) {          // one is found: pos < total
            const int places = b0 + lane < p.B ? places_of(b0 + lane) : 0, n = places * p.Hkv;
            int x = n;                              // inclusive prefix sum
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, run.pos < off + x);
            if (past) {
                const int l = __ffs(past) - 1;      // first sequence that ends past pos
                const int each = __shfl_sync(0xffffffffu, places, l);
                run.b = b0 + l;
                off += __shfl_sync(0xffffffffu, x - n, l);
                run.kvh = (run.pos - off) / each;
                run.tile0 = off + run.kvh * each + kD8Begin;
                break;
            }
            off += __shfl_sync(0xffffffffu, x, 31);
        }
    const uint32_t ring_addr = smem_u32(smem + warp * Lay::kRingBytes), bar_addr = smem_u32(full_bar[warp]);
    // where this thread reads a tile: K key d8_key(nb, gq), V key d8_key(k >> 1, 2 tq + (k & 1))
    uint32_t k_off[2][D / 64], v_off[4];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            k_off[nb][c] = d8_off<D>(d8_key<D>(nb, gq), tq * (D / 64) + c);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v_off[k] = d8_off<D>(d8_key<D>(k >> 1, 2 * tq + (k & 1)), D == 128 ? gq : gq >> 1) +
                   (D == 128 ? 0 : (gq & 1) * 8);

    __shared__ float2 rope_cs[kRope ? D / 2 : 1];
    int rope_len = INT_MIN;                         // the length whose turns it holds
    int st = 0;                                     // the warp's place in its ring, and its phase
    uint32_t ph = 0;
    // (b < B holds by the sums above; it is checked so that lengths which change under
    // the kernel can end the run early, but not lead it astray)
    while (run.pos < run.end && run.b < p.B) {
        const int b = run.b, len = p.seqlens[b], L = min(max(len, 0), Lmax);
        const D8Tiles seq(L, p.window, p.sinks);
        if (seq.n == 0) {
            ++run.b;
            continue;
        }
        const D8Piece piece = d8_take(run, seq.n, p.Hkv, per, blockIdx.x, gridDim.x);
        const int head = piece.head, first = piece.first, count = piece.count;
        const int cta0 = piece.cta0, cta1 = piece.cta1;
        const size_t unit = static_cast<size_t>(b) * p.Hkv + head;
        const size_t grow0 = unit * (p.Hq / p.Hkv) + blockIdx.y * p.share;
        const int32_t *row = p.table + static_cast<size_t>(b) * p.M;
        if (count <= 0) continue;
        const int n_iter = (count - warp + kD8Warps - 1) / kD8Warps;      // tiles of this warp
        auto key_of = [&](int t) { return seq.tile(first + warp + t * kD8Warps) * kD8Keys; };
        auto seen = [&](int key0, int n) {          // any of n keys visible
            return key0 < L && (key0 + n > seq.lo || key0 < seq.sinks);
        };
        // Lane i holds what is known of the 16 keys that are half i & 1 of tile i >> 1 of
        // an epoch: their first row in the cache (-1: not there; fits an int, checked on
        // the host), the place of their scales, and these.  The V scale is negated where
        // some of the keys are out of sight, and -inf where none is there.
        struct Group {
            int row, at;
            float ks, vs;
        };
        auto load_rows = [&](int epoch, Group &g) {
            const int t = epoch * kD8Epoch + (lane >> 1);
            const int key = key_of(t) + (lane & 1) * 16;
            g.row = -1;
            if (t < n_iter && seen(key, 16)) {      // key < L: the slot exists
                // key / 16 < 2^27 and page / 16 <= 64: the product is exact enough
                const int slot = static_cast<int>((static_cast<uint32_t>(key) >> 4) * p.page_inv >> 35);
                const int page = row[slot], off = key - slot * p.page;
                if (page >= 0 && page < p.n_pages) {
                    const int ph = page * p.Hkv + head;
                    g.row = ph * p.page + off;
                    g.at = ph * p.nblk + static_cast<int>((static_cast<uint32_t>(off) >> 4) * p.block_inv >> 16);
                } else {
                    record_status(p.status, GQA_ERR_INVALID_ARG);
                }
            }
        };
        auto load_scales = [&](int epoch, Group &g) {
            g.ks = 0.0f;
            g.vs = -INFINITY;
            if (g.row >= 0) {
                const int key = key_of(epoch * kD8Epoch + (lane >> 1)) + (lane & 1) * 16;
                g.ks = p.k_scale[g.at];
                g.vs = p.v_scale[g.at];
                if (!(key + 16 <= L && (key >= seq.lo || key + 16 <= seq.sinks))) g.vs = -g.vs;
            }
        };
        // Copies of tile t into ring slot sl, counted on the slot's barrier, by the lane
        // that holds the tile's first half; g: the groups of t's epoch.
        auto issue = [&](int t, int sl, int row0) {
            const int row1 = __shfl_down_sync(0xffffffffu, row0, 1);
            if (lane == (2 * t & 31)) {
                const uint32_t bar = bar_addr + sl * 8, kt = ring_addr + sl * Lay::kStageBytes;
                if (p.box == kD8Keys) {             // both halves lie in one page
                    const int r = max(row0, row1 - 16);
                    const bool there = max(row0, row1) >= 0;
                    mbar_expect_tx(&full_bar[warp][sl], there ? Lay::kStageBytes : 0);
                    if (there) {
                        copy_rows(kt, &tm_k, bar, r / (128 / D));
                        copy_rows(kt + Lay::kTileBytes, &tm_v, bar, r / (128 / D));
                    }
                } else {
                    mbar_expect_tx(&full_bar[warp][sl],
                                   ((row0 >= 0) + (row1 >= 0)) * (Lay::kStageBytes / 2));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = x ? row1 : row0;
                        if (r < 0) continue;
                        const uint32_t dst = kt + x * (Lay::kTileBytes / 2);
                        copy_rows(dst, &tm_k, bar, r / (128 / D));
                        copy_rows(dst + Lay::kTileBytes, &tm_v, bar, r / (128 / D));
                    }
                }
            }
            __syncwarp();
        };
        const D8Word word = word_of(unit);
        unsigned long long left = 0;
        if (threadIdx.x == 0 && cta0 != cta1) left = word.read();
        // Loads that nothing waits for yet come first: once the copies of all CTAs are
        // under way, a load takes several microseconds.
        Group cur, next;
        load_rows(0, cur);
        load_rows(1, next);
        // Query fragments (column gq of head tile nt).  Contraction step s multiplies
        // elements 4 s .. 4 s + 3 of each thread's quarter of the row (D / 4 elements).
        // One head tile is kept in registers; of more, each warp prepares one for all.
        constexpr int kQ = D / 4;
        const int own = NT == 1 ? 0 : warp, own_row = own * 8 + gq;
        const __nv_bfloat16 *qg = p.q + (grow0 + own_row) * D + tq * kQ;
        uint32_t qb[D / 16][2];
#pragma unroll
        for (int s = 0; s < D / 16; s += 2) {
            const uint4 w = own_row < G ? *reinterpret_cast<const uint4 *>(qg + 4 * s)
                                        : make_uint4(0u, 0u, 0u, 0u);
            qb[s][0] = w.x;
            qb[s][1] = w.y;
            qb[s + 1][0] = w.z;
            qb[s + 1][1] = w.w;
        }
        const bool turn = kRope && rope_len != len; // else they are the last piece's
        if (turn) {
            __syncthreads();                        // the last piece's turns are read
            rope_len = len;
            const int m = max(len - 1, 0);
            for (int i = threadIdx.x; i < D / 2; i += kD8Threads) {
                float cs, sn;
                rope_cos_sin(m, rope_turn[i], cs, sn);
                rope_cs[i] = make_float2(cs, sn);
            }
        }
        load_scales(0, cur);
        for (int t = 0; t < min(n_iter, kStages); ++t)
            issue(t, st + t < kStages ? st + t : st + t - kStages, cur.row);
        if (threadIdx.x == 0 && cta0 != cta1) d8_claim(word, left, p.call_id);
        if constexpr (kRope) {
            if (turn) __syncthreads();
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const float2 c0 = rope_cs[tq * (kQ / 2) + 2 * s];
                const float2 c1 = rope_cs[tq * (kQ / 2) + 2 * s + 1];
                qb[s][0] = rope_rotate_pair(qb[s][0], c0.x, c0.y);
                qb[s][1] = rope_rotate_pair(qb[s][1], c1.x, c1.y);
            }
        }
        // bring the row's largest value into [1, 2), a subnormal one near it; an infinite row stays
        // as it is
        float q_max = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const float2 a = bf16x2_to_float2(qb[s][0]), c = bf16x2_to_float2(qb[s][1]);
            q_max = fmaxf(q_max, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(c.x), fabsf(c.y))));
        }
        q_max = fmaxf(q_max, __shfl_xor_sync(0xffffffffu, q_max, 1));
        q_max = fmaxf(q_max, __shfl_xor_sync(0xffffffffu, q_max, 2));
        const int q_exp = static_cast<int>(__float_as_uint(q_max) >> 23);   // biased exponent
        const bool fit = q_exp < 255;
        const uint32_t ex = min(max(q_exp, 1), 253);    // 2^(ex - 127) and its inverse are normal
        const float up = fit ? __uint_as_float((254 - ex) << 23) : 1.0f;
        const float down = (fit ? __uint_as_float(ex << 23) : 1.0f) * p.scale_log2;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 a = bf16x2_to_float2(qb[s][h]);
                qb[s][h] = pack_f16x2(a.x * up, a.y * up);
            }
        float2 qs[NT];                                  // score scale of heads 2 tq, 2 tq + 1
        __shared__ uint4 q_tiles[NT == 1 ? 1 : NT][D / 32][32];      // steps s, s + 1 of a lane
        __shared__ float2 q_down[NT == 1 ? 1 : NT][4];
        if constexpr (NT == 1) {
            qs[0].x = __shfl_sync(0xffffffffu, down, 8 * tq);
            qs[0].y = __shfl_sync(0xffffffffu, down, 8 * tq + 4);
        } else {
            if (own < NT) {                             // (the last piece's tiles have been read)
#pragma unroll
                for (int s = 0; s < D / 16; s += 2)
                    q_tiles[own][s / 2][lane] = make_uint4(qb[s][0], qb[s][1], qb[s + 1][0], qb[s + 1][1]);
                if (tq == 0) reinterpret_cast<float *>(q_down[own])[gq] = down;
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) qs[nt] = q_down[nt][tq];
        }
        // O^T: product j, accumulator e is element (D / 8) gq + 2 j + (e >> 1) of head 2 tq + (e & 1)
        float oacc[NT][D / 16][4];
        float2 m_ref[NT], l_run[NT];                    // of heads 2 tq, 2 tq + 1
        float vref = -1.0f, vinv = 0.0f;                // O is in units of vref (-1: O is still 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[nt][j][e] = 0.0f;
            m_ref[nt] = make_float2(kD8Least, kD8Least);
            l_run[nt] = make_float2(0.0f, 0.0f);
        }

        bool ok = true;
        int t = 0;
        for (; t < n_iter; ++t) {
            // warp-uniform outcome: the products below are warp-collective
            ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[warp][st], ph, &abort_flag[warp], p.status));
            if (!ok) break;
            const uint32_t kt = ring_addr + st * Lay::kStageBytes;
            // the next epoch's rows are loaded one epoch ahead, its scales half of one
            if (t % kD8Epoch == kD8Epoch / 2) load_scales(t / kD8Epoch + 1, next);
            if (t % kD8Epoch == 0 && t > 0) {
                cur = next;
                load_rows(t / kD8Epoch + 1, next);
            }
            float ks[2], vs[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ks[x] = __shfl_sync(0xffffffffu, cur.ks, (2 * t + x) & 31);
                vs[x] = __shfl_sync(0xffffffffu, cur.vs, (2 * t + x) & 31);
            }
            // ---- S^T = K Q^T: half x, accumulator e is key (e >> 1, gq), head 2 tq + (e & 1) ----
            float sacc[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sacc[nt][x][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t w[2][2][4];                // [half][nb]
                lds<0>(w[0][0], kt + k_off[0][c]);
                lds<0>(w[0][1], kt + k_off[1][c]);
                lds<16 * D>(w[1][0], kt + k_off[0][c]);
                lds<16 * D>(w[1][1], kt + k_off[1][c]);
#pragma unroll
                for (int i0 = 0; i0 < 4; i0 += 2) {
                    uint4 q[NT];                    // steps i0 and i0 + 1
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int s = c * 4 + i0;
                        q[nt] = NT == 1 ? make_uint4(qb[s][0], qb[s][1], qb[s + 1][0], qb[s + 1][1])
                                        : q_tiles[nt][s / 2][lane];
                    }
#pragma unroll
                    for (int i = i0; i < i0 + 2; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t a[4];
                            to_f16x2<kInt8>(w[x][0][i], a[0], a[2]);
                            to_f16x2<kInt8>(w[x][1][i], a[1], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816_f16(sacc[nt][x], a, i == i0 ? q[nt].x : q[nt].z,
                                              i == i0 ? q[nt].y : q[nt].w);
                        }
                }
            }
            // ---- V scales: weight factor of each half, and O's change of units before it;
            //      keys out of sight: a bit of hide_k for half x, key (nb, gq) at 2 x + nb, of
            //      hide_v for its key (k >> 1, 2 tq + (k & 1)) at 4 x + k ----
            float pscale[2], ratio[2] = {1.0f, 1.0f};
            uint32_t hide_k = 0, hide_v = 0;
            if (vs[0] <= vref && vs[0] * 64.0f >= vref && vs[1] <= vref && vs[1] * 64.0f >= vref) {
                pscale[0] = vs[0] * vinv;           // all in sight: vref is positive or -1
                pscale[1] = vs[1] * vinv;
            } else {
                const int key0 = key_of(t);
                auto hidden = [&](int x, int nb, int n) -> uint32_t {
                    const int key = key0 + x * 16 + d8_key<D>(nb, n);
                    return vs[x] == -INFINITY || key >= L || (key < seq.lo && key >= seq.sinks);
                };
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (signbit(vs[x])) {
#pragma unroll
                        for (int nb = 0; nb < 2; ++nb) hide_k |= hidden(x, nb, gq) << (2 * x + nb);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            hide_v |= hidden(x, k >> 1, 2 * tq + (k & 1)) << (4 * x + k);
                    }
                    const float v = fabsf(vs[x]);
                    pscale[x] = 0.0f;               // scale 0, or not there
                    if (v == 0.0f || vs[x] == -INFINITY) continue;
                    if (!(v <= vref && v * 64.0f >= vref)) {
                        if (v < vref) {             // a smaller unit, as far as O has room
                            float top = largest(oacc);
                            if (x == 1) top = top * ratio[0] + kD8HalfTop;
                            ratio[x] = fminf(vref / v, fmaxf(kD8Room / fmaxf(top, kD8Room * 0x1p-126f), 1.0f));
                            vref /= ratio[x];
                        } else {
                            if (vref > 0.0f) ratio[x] = vref / v;
                            vref = v;
                        }
                        vinv = 1.0f / vref;
                    }
                    pscale[x] = v * vinv;
                }
            }
            float2 f[NT][2];                        // factor of the scores of heads 2 tq, 2 tq + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) f[nt][x] = mul2(qs[nt], make_float2(ks[x], ks[x]));
            if (hide_k) {
                // -inf must stay so whatever its factor: the scores are scaled here
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sacc[nt][x][e] *= e & 1 ? f[nt][x].y : f[nt][x].x;
                            if (hide_k >> (2 * x + (e >> 1)) & 1) sacc[nt][x][e] = -INFINITY;
                        }
                        f[nt][x] = make_float2(1.0f, 1.0f);
                    }
            }
            // ---- softmax: the reference m only moves when a score passes it by more than
            //      kD8Rescale, so that O and l are seldom rescaled ----
            auto rescale = [&](int nt, float f0, float f1) {
                const float2 f = make_float2(f0, f1);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int h = 0; h < 4; h += 2) {
                        const float2 o = mul2(make_float2(oacc[nt][j][h], oacc[nt][j][h + 1]), f);
                        oacc[nt][j][h] = o.x;
                        oacc[nt][j][h + 1] = o.y;
                    }
            };
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float(&s)[2][4] = sacc[nt];
                float mx[2];
                mx[0] = fmaxf(fmaxf(s[0][0], s[0][2]) * f[nt][0].x, fmaxf(s[1][0], s[1][2]) * f[nt][1].x);
                mx[1] = fmaxf(fmaxf(s[0][1], s[0][3]) * f[nt][0].y, fmaxf(s[1][1], s[1][3]) * f[nt][1].y);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 4));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 8));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
                }
                if (__any_sync(0xffffffffu, mx[0] > m_ref[nt].x + kD8Rescale ||
                                                mx[1] > m_ref[nt].y + kD8Rescale)) {
                    const float2 m = make_float2(fmaxf(m_ref[nt].x, mx[0]), fmaxf(m_ref[nt].y, mx[1]));
                    const float2 alpha = make_float2(fast_exp2(m_ref[nt].x - m.x),
                                                     fast_exp2(m_ref[nt].y - m.y));
                    m_ref[nt] = m;
                    l_run[nt] = mul2(l_run[nt], alpha);
                    rescale(nt, alpha.x, alpha.y);
                }
                const float2 minus_m = make_float2(kD8Lift - m_ref[nt].x, kD8Lift - m_ref[nt].y);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        float2 w = fma2(make_float2(s[x][2 * nb], s[x][2 * nb + 1]), f[nt][x], minus_m);
                        w = make_float2(fast_exp2(w.x), fast_exp2(w.y));
                        l_run[nt] = add2(l_run[nt], w);
                        w = mul2(w, make_float2(pscale[x], pscale[x]));
                        pb[nt][x][nb] = transpose_8x8(pack_f16x2(w.x, w.y));
                    }
            }
            // ---- O^T += V^T P^T ----
            constexpr int kW = D / 32;              // words of V per key and thread
            uint32_t vw[2][4][kW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lds<Lay::kTileBytes>(vw[0][k], kt + v_off[k]);
                lds<Lay::kTileBytes + 16 * D>(vw[1][k], kt + v_off[k]);
            }
            if (hide_v) {
                // rows out of sight hold anything, NaN included: 0 weight times 0
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int w = 0; w < kW; ++w)
                            if (hide_v >> (4 * x + k) & 1) vw[x][k][w] = 0u;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (ratio[x] != 1.0f)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) rescale(nt, ratio[x], ratio[x]);
#pragma unroll
                for (int w = 0; w < kW; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // elements 4 w + 2 h, 4 w + 2 h + 1
                        const uint32_t sel = h ? 0x7362 : 0x5140;
                        uint32_t a[4];
                        to_f16x2<kInt8>(__byte_perm(vw[x][0][w], vw[x][1][w], sel), a[0], a[1]);
                        to_f16x2<kInt8>(__byte_perm(vw[x][2][w], vw[x][3][w], sel), a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816_f16(oacc[nt][2 * w + h], a, pb[nt][x][0], pb[nt][x][1]);
                    }
            }
            __syncwarp();                               // the slot is read: refill it
            if (t + kStages < n_iter)
                issue(t + kStages, st, (t + kStages) / kD8Epoch == t / kD8Epoch ? cur.row : next.row);
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
        }
        // after a time-out, the copies in flight land before the block exits
        if (!ok)
            for (int u = t; u < min(n_iter, t + kStages); ++u) {
                mbar_drain(&full_bar[warp][st], ph, p.status);
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }

        // ---- merge the four warps' partial softmax states ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                l_run[nt].x += __shfl_xor_sync(0xffffffffu, l_run[nt].x, x);
                l_run[nt].y += __shfl_xor_sync(0xffffffffu, l_run[nt].y, x);
            }
        if (lane == 0) s_vref[warp] = fmaxf(vref, 0.0f);
        __syncthreads();                                // every tile consumed: reuse the rings
        if (abort_flag[0] | abort_flag[1] | abort_flag[2] | abort_flag[3]) {
            if (threadIdx.x == 0) {                     // a replay finds the words as it needs them
                if (cta0 != cta1) d8_arrive(word, cta1 - cta0 + 1, p.call_id);
                d8_abandon(run, p.B, p.Hkv, per, blockIdx.x, gridDim.x, p.call_id,
                           [&](int z) { return max(places_of(z) - kD8Begin, 0); },
                           [&](int z, int h) { return word_of(static_cast<size_t>(z) * p.Hkv + h); });
            }
            return;
        }
        constexpr int kRows = Lay::kRows, kStride = Lay::kRowFloats;
        float *s_o = reinterpret_cast<float *>(smem);             // [warp][row][kStride]
        float *s_m = s_o + kD8Warps * kRows * kStride;            // [warp][row]
        float *s_l = s_m + kD8Warps * kRows;                      // [warp][row]
        auto column = [](int c) { return c + 4 * (c / (D / 8)); };
        // Sums of large values may be past fp32's range although their mean is not, so the
        // rows stay in units of their warp's vref: v_rel takes these to v_unit, a power of two
        // near the largest, which the mean is multiplied by.
        const float4 v_of = *reinterpret_cast<const float4 *>(s_vref);
        const float v_top = fmaxf(fmaxf(v_of.x, v_of.y), fmaxf(v_of.z, v_of.w));
        const uint32_t v_exp = min(max(__float_as_uint(v_top) >> 23, 1u), 253u);   // unit and inverse are normal
        const float v_unit = __uint_as_float(v_exp << 23), v_inv = __uint_as_float((254 - v_exp) << 23);
        const float v_rel[kD8Warps] = {v_of.x * v_inv, v_of.y * v_inv, v_of.z * v_inv, v_of.w * v_inv};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = nt * 8 + 2 * tq + h;
                float *dst = s_o + (warp * kRows + r) * kStride + column((D / 8) * gq);
#pragma unroll
                for (int j = 0; j < D / 16; j += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * j) =
                        make_float4(oacc[nt][j][h], oacc[nt][j][h + 2], oacc[nt][j + 1][h], oacc[nt][j + 1][h + 2]);
                if (gq == 0) {
                    s_m[warp * kRows + r] = h ? m_ref[nt].y : m_ref[nt].x;
                    s_l[warp * kRows + r] = h ? l_run[nt].y : l_run[nt].x;
                }
            }
        __syncthreads();
        for (int idx = threadIdx.x; idx < G * D / 4; idx += kD8Threads) {
            const int r = idx / (D / 4), c = idx % (D / 4) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kD8Warps; ++w) M = fmaxf(M, s_m[w * kRows + r]);
            float wsum = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kD8Warps; ++w) {
                const float f = fast_exp2(s_m[w * kRows + r] - M);
                const float4 x =
                    *reinterpret_cast<const float4 *>(s_o + (w * kRows + r) * kStride + column(c));
                const float g = f * v_rel[w];
                wsum += f * s_l[w * kRows + r];
                acc.x += g * x.x;
                acc.y += g * x.y;
                acc.z += g * x.z;
                acc.w += g * x.w;
            }
            const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
            acc = make_float4(acc.x * inv * v_unit, acc.y * inv * v_unit, acc.z * inv * v_unit,
                              acc.w * inv * v_unit);
            if (cta0 == cta1) {
                *reinterpret_cast<uint2 *>(p.o + (grow0 + r) * D + c) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            } else {
                // slot 0 of the CTA: a unit that an earlier run began; slot 1: begun here
                const size_t at = (2 * static_cast<size_t>(cta) + (first == 0)) * p.share + r;
                *reinterpret_cast<float4 *>(p.part_o + at * D + c) = acc;
                if (c == 0) p.part_lse[at] = wsum == 0.0f ? -INFINITY : M + __log2f(wsum);
            }
        }
        // the rings held plain data: order it before the next piece's copies
        fence_proxy_async_smem();
        if (cta0 == cta1) {
            __syncthreads();
            continue;
        }

        // ---- the last piece of the unit to arrive merges all of them ----
        __syncthreads();                            // the piece's rows are written
        const int pieces = cta1 - cta0 + 1;
        if (threadIdx.x == 0) {
            // releases the CTA's rows (ordered before by the barrier) and acquires the others'
            merger = d8_arrive(word, pieces, p.call_id);
        }
        __syncthreads();
        if (!merger) continue;
        // One or two head rows per warp at a time, D / 4 lanes for a row's columns; the other half
        // of the warp (D = 64) takes every second piece.  The maximum runs over batches of
        // pieces, whose lse and rows are loaded together.
        constexpr int kLanes = D / 4, kSub = 32 / kLanes, kBatch = 8;
        const int sub = lane / kLanes, c = lane % kLanes * 4;
        // rows of piece i: slot 1 of the first CTA, slot 0 of the others
        const int slot0 = blockIdx.y * gridDim.x + cta0;
        auto slot = [&](int i) { return (2 * (slot0 + i) + (i == 0)) * p.share; };
        auto merge_rows = [&](int r0, auto count) {
            constexpr int kR = decltype(count)::value;
            float M[kR], wsum[kR];
            float4 acc[kR];
#pragma unroll
            for (int y = 0; y < kR; ++y) {
                M[y] = kD8Least;                    // finite: a piece of lse NaN has weight NaN
                wsum[y] = 0.0f;
                acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            for (int i = 0; i < pieces; i += kSub * kBatch) {
                float l[kR][kBatch];
                float4 v[kR][kBatch];
#pragma unroll
                for (int y = 0; y < kR; ++y)
#pragma unroll
                    for (int x = 0; x < kBatch; ++x) {
                        const int at = i + x * kSub + sub;
                        const bool in = at < pieces;
                        const size_t row = slot(at) + r0 + y * kD8Warps;
                        l[y][x] = in ? __ldcg(p.part_lse + row) : -INFINITY;
                        v[y][x] = in ? __ldcg(reinterpret_cast<const float4 *>(p.part_o + row * D + c))
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                for (int y = 0; y < kR; ++y) {
                    float m = M[y];
#pragma unroll
                    for (int x = 0; x < kBatch; ++x) m = fmaxf(m, l[y][x]);
                    if constexpr (kSub == 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const float f = fast_exp2(M[y] - m);
                    M[y] = m;
                    m += kD8Pieces;
                    wsum[y] *= f;
                    float4 a = make_float4(acc[y].x * f, acc[y].y * f, acc[y].z * f, acc[y].w * f);
#pragma unroll
                    for (int x = 0; x < kBatch; ++x) {
                        const float w = fast_exp2(l[y][x] - m);
                        wsum[y] += w;
                        a.x += w * v[y][x].x;
                        a.y += w * v[y][x].y;
                        a.z += w * v[y][x].z;
                        a.w += w * v[y][x].w;
                    }
                    acc[y] = a;
                }
            }
#pragma unroll
            for (int y = 0; y < kR; ++y) {
                float4 a = acc[y];
                if constexpr (kSub == 2) {
                    wsum[y] += __shfl_xor_sync(0xffffffffu, wsum[y], 16);
                    a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
                    a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
                    a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
                    a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
                }
                const float inv = wsum[y] == 0.0f ? 0.0f : 1.0f / wsum[y];
                if (sub == 0)
                    *reinterpret_cast<uint2 *>(p.o + (grow0 + r0 + y * kD8Warps) * D + c) = make_uint2(
                        pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            }
        };
        for (int r = warp; r < G;) {                // (four rows would spill)
            if (r + kD8Warps < G) {
                merge_rows(r, std::integral_constant<int, 2>{});
                r += 2 * kD8Warps;
            } else {
                merge_rows(r, std::integral_constant<int, 1>{});
                r += kD8Warps;
            }
        }
        __syncthreads();                            // merger is read
    }
    // sequences without a visible key: zeros; lengths outside the table: flagged
    for (int z = cta; z < p.B; z += gridDim.x * gridDim.y) {
        if (threadIdx.x == 0 && (p.seqlens[z] < 0 || p.seqlens[z] > Lmax))
            record_status(p.status, GQA_ERR_INVALID_ARG);
        if (places_of(z) == 0)
            for (int i = threadIdx.x; i < p.Hq * D / 8; i += kD8Threads)
                reinterpret_cast<uint4 *>(p.o + static_cast<size_t>(z) * p.Hq * D)[i] =
                    make_uint4(0u, 0u, 0u, 0u);
    }
}

static long long d8_tiles(long long keys) { return (keys + kD8Keys - 1) / kD8Keys; }

// CTAs that B sequences of up to `tiles` tiles can keep busy, at most `most`.
static int d8_grid(int B, int Hkv, long long tiles, int most) {
    const double runs = ceil(static_cast<double>(tiles + kD8Begin) * B * Hkv / kD8MinTiles);
    return runs < most ? static_cast<int>(runs) : most;
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// CTAs that split the heads of a group, and the heads that each takes.
static int d8_groups(int G) { return (G + kD8Heads - 1) / kD8Heads; }
static int d8_share(int G) { return (G - 1) / d8_groups(G) + 1; }

// Workspace: partial O [CTAs, 2, heads per CTA, d] fp32 | partial lse [CTAs, 2, heads per
// CTA] fp32 (log2 units) | arrival words [B, Hkv, CTAs of a group] u64.
struct D8Workspace {
    size_t off_lse, off_arrivals, bytes;
    D8Workspace(int B, int Hq, int Hkv, int d, long long Lmax) {
        const int G = Hq / Hkv, groups = d8_groups(G);
        const size_t ctas = static_cast<size_t>(d8_grid(B, Hkv, d8_tiles(Lmax), kD8MaxCtas / groups)) * groups;
        const size_t rows = ctas * 2 * d8_share(G);
        off_lse = align256(rows * d * sizeof(float));
        off_arrivals = off_lse + align256(rows * sizeof(float));
        bytes = off_arrivals + align256(static_cast<size_t>(B) * Hkv * groups * 8);
    }
};

template <int D, int NT, bool kInt8, bool kRope>
static int launch_decode8_kernel(const CUtensorMap &tk, const CUtensorMap &tv, const D8Params &p,
                                 long long tiles, cudaStream_t stream) {
    auto kern = decode8_kernel<D, NT, kInt8, kRope>;
    const int smem = D8Layout<D, NT>::kSmemBytes;
    static CtxSlot setup;   // one per instantiation: the opt-in is set once per context
    if (int rc = once_per_context(setup, [&](int) {
            return check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   smem), "cudaFuncSetAttribute(decode8)");
        }))
        return rc;
    int n_sm = 0;
    if (int rc = sm_count(&n_sm)) return rc;
    const int groups = d8_groups(p.Hq / p.Hkv);
    const int most = min(kD8MaxCtas, n_sm * kD8CtasPerSm) / groups;    // all resident at once
    return launch_dependent(kern, dim3(d8_grid(p.B, p.Hkv, tiles, most), groups), kD8Threads, smem, stream,
                            "decode8_kernel launch", tk, tv, p);
}

template <int D, int NT>
static int launch_decode8_kind(bool int8, bool rope, const CUtensorMap &tk, const CUtensorMap &tv,
                               const D8Params &p, long long tiles, cudaStream_t s) {
    if (int8)
        return rope ? launch_decode8_kernel<D, NT, true, true>(tk, tv, p, tiles, s)
                    : launch_decode8_kernel<D, NT, true, false>(tk, tv, p, tiles, s);
    return rope ? launch_decode8_kernel<D, NT, false, true>(tk, tv, p, tiles, s)
                : launch_decode8_kernel<D, NT, false, false>(tk, tv, p, tiles, s);
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
    if (B == 0) return GQA_OK;
    // a windowed sequence reads the tiles of its sinks and of its window
    long long tiles = d8_tiles(static_cast<long long>(M) * page);
    if (window > 0 && d8_tiles(window) + 1 + d8_tiles(sinks) < tiles)
        tiles = d8_tiles(window) + 1 + d8_tiles(sinks);
    if (static_cast<double>(tiles + kD8Begin) * B * Hkv > 2147483647.0 - kD8MaxCtas)
        return set_error(GQA_ERR_UNSUPPORTED, "decode8: B=%d x Hkv=%d x M=%d x page=%d rows are too many", B,
                         Hkv, M, page);
    if (int rc = check_ptr(q, 16, "q")) return rc;
    if (int rc = check_ptr(o, 16, "o")) return rc;
    if (int rc = check_ptr(table, 4, "table")) return rc;
    if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
    const D8Workspace ws(B, Hq, Hkv, d, static_cast<long long>(M) * page);
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
    p.share = d8_share(Hq / Hkv);
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.M = M;
    p.n_pages = n_pages;
    p.page = page;
    p.page_inv = ((1ull << 35) + page / 16 - 1) / (page / 16);
    p.block_inv = ((1u << 16) + block / 16 - 1) / (block / 16);
    p.nblk = page / block;
    p.box = page % kD8Keys == 0 ? kD8Keys : 16;
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
    if (d == 128)
        return p.share <= 8 ? launch_decode8_kind<128, 1>(int8, rope, tk, tv, p, tiles, s)
                            : launch_decode8_kind<128, 2>(int8, rope, tk, tv, p, tiles, s);
    return p.share <= 8 ? launch_decode8_kind<64, 1>(int8, rope, tk, tv, p, tiles, s)
                        : launch_decode8_kind<64, 2>(int8, rope, tk, tv, p, tiles, s);
}
